"""What the stand-alone operators refuse, before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def B():
    from latentmoe_expert_routing_b200 import build
    build.build()
    from latentmoe_expert_routing_b200 import binding
    return binding


P = 4096                                   # aligned, never dereferenced
inf, nan = float("inf"), float("nan")


def _topk(B, **kw):
    a = dict(logits=P, dtype=0, ld=64, bias=P, T=4, E=64, k=8, score=0, n_group=1, topk_group=1,
             renorm=1, scale=1.0, idx=P, w=P)
    a.update(kw)
    return B.lib.moe_route_topk(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=65, E=64), 1), (dict(ld=63), 1),
    (dict(dtype=2), 1), (dict(score=2), 1), (dict(scale=inf), 1), (dict(scale=nan), 1),
    (dict(n_group=0), 1), (dict(topk_group=0), 1), (dict(n_group=4, topk_group=5), 1),
    (dict(n_group=3), 1), (dict(n_group=64), 1), (dict(n_group=16, topk_group=1), 1),
    (dict(logits=None), 1), (dict(idx=None), 1), (dict(w=None), 1), (dict(logits=P + 2), 1),
    (dict(bias=P + 1), 1), (dict(E=1025, ld=1025), 2), (dict(E=128, ld=128, k=65), 2),
    (dict(E=256, ld=256, n_group=128, topk_group=8), 2), (dict(T=0, logits=None, idx=None, w=None), 0),
])
def test_route_topk_refuses(B, kw, status):
    assert _topk(B, **kw) == status


def _topk_bwd(B, **kw):
    a = dict(logits=P, dtype=0, ld=64, idx=P, w=P, dw=P, T=4, E=64, k=8, score=0, renorm=1,
             scale=1.0, dl=P, ldd=64)
    a.update(kw)
    return B.lib.moe_route_topk_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(ldd=63), 1), (dict(dl=None), 1), (dict(dw=None), 1), (dict(w=None), 1),
    (dict(idx=None), 1), (dict(scale=nan), 1), (dict(k=65, E=128, ld=128, ldd=128), 2),
    (dict(T=0, dl=None), 0),
])
def test_route_topk_backward_refuses(B, kw, status):
    assert _topk_bwd(B, **kw) == status


def test_route_group_refuses(B):
    f, need = B.lib.moe_route_group, B.moe_route_group_workspace
    n = need(100, 8, 64)
    assert n == 64 * 4 and need(-1, 8, 64) == 0 and need(4, 0, 64) == 0
    assert f(P, 100, 8, 64, P, P, P, P, P, n - 1, None) == INVALID       # workspace too small
    assert f(P, 100, 8, 64, P, P, P, P, P + 4, n, None) == INVALID
    assert f(P, 100, 8, 64, P, P, P, P, None, n, None) == INVALID
    assert f(None, 100, 8, 64, P, P, P, P, P, n, None) == INVALID
    assert f(P, 100, 8, 64, None, P, P, P, P, n, None) == INVALID
    assert f(P, 100, 8, 0, P, P, P, P, P, n, None) == INVALID
    assert f(P, 1 << 30, 8, 64, P, P, P, P, P, 1 << 40, None) == INVALID  # pair ids are 32-bit
    assert f(P, 100, 8, 1025, P, P, P, P, P, 1 << 20, None) == UNSUPPORTED


def _norm(B, **kw):
    a = B.moe_norm_args(T=4, D=64, dtype=1, gate_kind=1, residual_scale=1.0, eps=1e-5, x=P, ldx=64,
                        y=P, ldy=64, post_weight=P, pre_weight=P, gate=P, ldg=64, r=P, ldr=64, h=P,
                        ldh=64, rstd_y=P, rstd_r=P, dr=P, lddr=64, dh=P, lddh=64, dx=P, lddx=64,
                        dy=P, lddy=64, dpost_weight=P, dpre_weight=P, dgate=P, lddg=64)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


BOTH = [
    (dict(T=-1), 1), (dict(D=0), 1), (dict(D=60), 1), (dict(dtype=3), 1), (dict(eps=0.0), 1),
    (dict(eps=inf), 1), (dict(eps=nan), 1), (dict(residual_scale=inf), 1), (dict(gate_kind=4), 1),
    (dict(gate=None), 1), (dict(gate_kind=3, ldg=63), 1), (dict(gate_kind=2, gate=P + 1), 1),
    (dict(y=None), 1), (dict(r=None), 1), (dict(ldy=63), 1), (dict(ldy=68), 1), (dict(y=P + 8), 1),
    (dict(post_weight=P + 2), 1), (dict(pre_weight=P + 2), 1), (dict(D=16392, ldy=1 << 15), 2),
]


@pytest.mark.parametrize("kw,status", BOTH + [(dict(x=None), 1), (dict(h=None), 1), (dict(ldh=60), 1),
                                              (dict(rstd_y=P + 2), 1), (dict(T=0, x=None, y=None), 0)])
def test_norm_refuses(B, kw, status):
    assert B.lib.moe_norm_residual(ctypes.byref(_norm(B, **kw)), None) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(dx=None), 1), (dict(dy=None), 1), (dict(dh=None), 1), (dict(dr=P + 4), 1),
    (dict(rstd_y=None), 1), (dict(rstd_r=None), 1), (dict(dpost_weight=None), 1),
    (dict(dpre_weight=None), 1), (dict(dgate=None), 1), (dict(gate_kind=2, dgate=None), 1),
    (dict(gate_kind=3, lddg=60), 1)])
def test_norm_backward_refuses(B, kw, status):
    n = B.moe_norm_residual_workspace(4, 64)
    assert n > 0
    assert B.lib.moe_norm_residual_backward(ctypes.byref(_norm(B, **kw)), P, n, None) == status


def test_norm_workspace_is_checked(B):
    a, n = _norm(B), B.moe_norm_residual_workspace(4, 64)
    f = B.lib.moe_norm_residual_backward
    assert f(ctypes.byref(a), P, n - 1, None) == INVALID
    assert f(ctypes.byref(a), None, n, None) == INVALID
    assert f(ctypes.byref(a), P + 8, n, None) == INVALID
    assert f(None, P, n, None) == INVALID and B.lib.moe_norm_residual(None, None) == INVALID
    assert B.moe_norm_residual_workspace(0, 64) == 0 and B.moe_norm_residual_workspace(4, -1) == 0


def test_quantize_refuses(B):
    def rows(x=P, dt=1, xr=8, K=256, ldx=256, perm=None, r=8, k=1, relu2=0, c=P, ldc=256, s=P, lds=8):
        return B.lib.moe_quantize_fp8(x, dt, xr, K, ldx, perm, r, k, relu2, c, ldc, s, lds, None)
    assert rows(r=0, xr=0) == 0
    for kw in (dict(K=0), dict(ldx=255), dict(dt=2), dict(r=7), dict(lds=7), dict(ldc=255), dict(ldc=264),
               dict(c=None), dict(c=P + 8), dict(s=None), dict(x=None), dict(x=P + 1), dict(perm=P, k=0),
               dict(xr=-1), dict(s=P + 1)):
        assert rows(**kw) == INVALID, kw

    def cols(x=P, dt=1, r=100, K=64, ldx=64, c=P, ldc=112, s=P, lds=64):
        return B.lib.moe_quantize_fp8_t(x, dt, r, K, ldx, c, ldc, s, lds, None)
    assert cols(r=0) == 0
    for kw in (dict(ldc=100), dict(ldc=96), dict(lds=63), dict(K=0), dict(x=None), dict(c=P + 4)):
        assert cols(**kw) == INVALID, kw

    def weight(w=P, dt=1, n=1, N=64, K=64, ldw=64, c=P, ldc=64, s=P, ct=None, ldct=64, st=None):
        return B.lib.moe_quantize_fp8_weight(w, dt, n, N, K, ldw, c, ldc, s, ct, ldct, st, None)
    for kw in (dict(w=None), dict(n=0), dict(N=0), dict(ldw=63), dict(ct=P), dict(st=P),
               dict(ct=P, st=P, ldct=63), dict(s=None), dict(c=None)):
        assert weight(**kw) == INVALID, kw


def test_gemm_refuses(B):
    def gemm(**kw):
        g = B.moe_fp8_gemm(M=8, N=64, K=256, n_groups=0, offsets=None, a=P, lda=256, a_scales=P,
                           lda_scales=8, b=P, ldb=256, b_scales=P, ldb_scales=0, out=P, ldo=64,
                           out_dtype=1)
        for n, v in kw.items():
            setattr(g, n, v)
        return B.lib.moe_gemm_fp8(ctypes.byref(g), None)
    assert gemm(M=0, a=None, out=None) == 0
    assert B.lib.moe_gemm_fp8(None, None) == INVALID
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(lda=240), dict(lda=264), dict(a=P + 8), dict(b=None),
               dict(ldb=240), dict(lda_scales=7), dict(ldb_scales=63), dict(ldb_scales=-1), dict(ldo=63),
               dict(out=P + 1), dict(out=None), dict(out_dtype=5), dict(a_scales=None), dict(b_scales=P + 2),
               dict(offsets=P, n_groups=0), dict(offsets=P, n_groups=2, ldb_scales=64),
               dict(offsets=P + 2, n_groups=2)):
        assert gemm(**kw) == INVALID, kw
    assert gemm(offsets=P, n_groups=1025) == UNSUPPORTED
    assert gemm(N=1 << 30, ldo=1 << 30, offsets=P, n_groups=4) == UNSUPPORTED


def test_python_layer_wants_cuda_tensors(B):
    from latentmoe_expert_routing_b200 import ops
    x, i = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    f8 = ops.Fp8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4))
    for call in (lambda: ops.route_topk(x, 2), lambda: ops.route_topk_backward(x, i, x, x),
                 lambda: ops.route_group(i, 4), lambda: ops.norm_residual(x, x),
                 lambda: ops.norm_residual_backward(x, None, x, ops.NormForward(x, None, None, None)),
                 lambda: ops.quantize_fp8(x), lambda: ops.quantize_fp8_weight(x),
                 lambda: ops.gemm_fp8(f8, f8)):
        with pytest.raises(ValueError, match="cuda"):
            call()


def test_struct_layout_matches_the_header(B, tmp_path):
    """The ctypes structures have the C structures' size and field offsets."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "latentmoe.h"', "int main(void) {"]
    for s in (B.moe_norm_args, B.moe_fp8_gemm):
        src.append(f'printf("%zu\\n", sizeof({s.__name__}));')
        src += [f'printf("%zu\\n", offsetof({s.__name__}, {f}));' for f, _ in s._fields_]
    (tmp_path / "t.c").write_text("\n".join(src) + "\nreturn 0; }\n")
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "t.c"), "-o",
                           str(tmp_path / "t")])
    got = [int(v) for v in subprocess.check_output([str(tmp_path / "t")]).split()]
    want = []
    for s in (B.moe_norm_args, B.moe_fp8_gemm):
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want
