"""Edges of the stand-alone operators' argument ranges, without a GPU."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from latentmoe_expert_routing_b200 import build
    build.build()
    from latentmoe_expert_routing_b200 import binding
    return binding


def test_workspace_queries_answer_every_size(B):
    """In a process of its own: a query must not end it."""
    code = ("from latentmoe_expert_routing_b200 import binding as B\n"
            "big = 2 ** 31 - 1\n"
            "for T in (-big, -1, 0, 1, 4, big):\n"
            "    for D in (-big, -1, 0, 1, 4, 7, 8, 12, 64, 16384, 16385, 16392, big):\n"
            "        n = B.moe_norm_residual_workspace(T, D)\n"
            "        ok = T > 0 and 0 < D <= 16384 and D % 8 == 0\n"
            "        assert (n > 0) == ok, (T, D, n)\n"
            "    for k in (-1, 0, 1, 64, big):\n"
            "        for E in (-1, 0, 1, 1024, big):\n"
            "            B.moe_route_group_workspace(T, k, E)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


def test_kernels_launched_early_read_with_ordinary_loads():
    """A kernel that may start while the one in front of it still writes its input
    must not promise that memory to be constant (non-coherent loads do)."""
    csrc = os.path.join(ROOT, "latentmoe_expert_routing_b200", "csrc")
    early = []
    for name in sorted(os.listdir(csrc)):
        text = open(os.path.join(csrc, name)).read()
        if name.endswith(".cu") and "after_previous();" in text:
            early.append(name)
            for word in ("__ldg", "__restrict__", "ld.global.nc"):
                assert word not in text, (name, word)
    assert {"umma_fp8.cu", "fp8_quant.cu", "route_ops.cu", "norm_ops.cu"} <= set(early)


def test_sizes_past_the_kernels_index_range_are_refused(B):
    """Addresses are never dereferenced: each call is refused before a launch."""
    P, top, unsupported = 4096, 2 ** 31 - 1, 2
    for K in (top, top - 1023):
        ld = (K + 15) // 16 * 16
        assert B.lib.moe_quantize_fp8(P, 1, 1, K, K, None, 1, 1, 0, P, ld, P, 1, None) == unsupported
    assert B.lib.moe_quantize_fp8_t(P, 1, 65535 * 128 + 1, 8, 8, P, 65536 * 128, P, 8, None) == unsupported
    assert B.lib.moe_quantize_fp8_weight(P, 1, 65536, 8, 8, 8, P, 16, P, None, 0, None, None) == unsupported
    K = 65535 * 128 + 1
    assert B.lib.moe_quantize_fp8_weight(P, 1, 1, 8, K, K, P, K + 15, P, None, 0, None, None) == unsupported
