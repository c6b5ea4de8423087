"""torch-facing wrappers of the library's stand-alone operators (marshalling only).

    idx, w = route_topk(logits, k, bias=b)                # scores, selection, weights
    counts, offsets, perm, pos = route_group(idx, E)      # pairs by expert
    z = quantize_fp8(x, perm=perm, k=k)                   # their rows as E4M3 codes
    h = gemm_fp8(z, up, offsets=offsets)                  # every expert's product
    y = gemm_fp8(quantize_fp8(h, relu2=True), down, offsets=offsets)
    f = norm_residual(x, y, ...)                          # f.r, f.h

Every function runs on the current stream of its tensors' device and returns new
tensors.  The gradients are calls of their own (route_topk_backward,
norm_residual_backward, and gemm_fp8 on transposed operands); nothing registers
with autograd.  Wrong arguments raise ValueError, a refusal by the library
MoeError.  What the C calls expect and promise stands in include/latentmoe.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B

_F32, _BF16, _I32, _F8 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn
_CODE = {_F32: B.MOE_FP32, _BF16: B.MOE_BF16}
_OUT = {"fp32": _F32, "bf16": _BF16}


class Fp8(NamedTuple):
    """E4M3 codes and their fp32 scales, one for each block of 128.

    rows (quantize_fp8):        codes [M, K], scales [ceil(K/128), M]
    weights (.._weight):        codes [N, K], scales [ceil(N/128), ceil(K/128)]
    experts' weights:           codes [E, N, K], scales [E, ceil(N/128), ceil(K/128)]

    codes are float8_e4m3fn (or their bytes as uint8), K innermost, in rows
    whose stride is a multiple of 16."""
    codes: torch.Tensor
    scales: torch.Tensor


class NormForward(NamedTuple):
    r: torch.Tensor
    h: Optional[torch.Tensor]
    rstd_y: Optional[torch.Tensor]
    rstd_r: Optional[torch.Tensor]


class NormBackward(NamedTuple):
    dx: torch.Tensor
    dy: torch.Tensor
    dpost_weight: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


class _on:
    """Makes the tensors' device current for a call; `_on(dev).stream` is its
    current stream."""

    def __init__(self, dev):
        self.dev, self.old = dev.index, torch.cuda.current_device()

    def __enter__(self):
        if self.dev != self.old:
            torch.cuda.set_device(self.dev)
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc):
        if self.dev != self.old:
            torch.cuda.set_device(self.old)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _dtype(t, what):
    _need(t.dtype in _CODE, f"{what} must be float32 or bfloat16")
    return _CODE[t.dtype]


def _same(dev, **tensors):
    for n, t in tensors.items():
        _need(t is None or t.device == dev, f"{n} must be on {dev}")


def _cuda(t, what):
    _need(isinstance(t, torch.Tensor) and t.is_cuda, f"{what} must be a cuda tensor")
    return t.device


def _rows(t):
    """t [R, C] with contiguous rows, and their stride; a copy where t's are not."""
    if t.stride(1) != 1 and t.shape[1] != 1 or t.stride(0) < t.shape[1] and t.shape[0] > 1:
        t = t.contiguous()
    return t, max(t.stride(0), t.shape[1])


def _rows16(t):
    """The same, each row starting on 16 bytes."""
    t, ld = _rows(t)
    if t.data_ptr() % 16 or ld * t.element_size() % 16:
        t = t.clone(memory_format=torch.contiguous_format)
        ld = t.shape[1]
    return t, ld


def _vec16(t):
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _up16(n):
    return (n + 15) // 16 * 16


def _blocks(n):
    return (n + 127) // 128


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def route_topk(logits, k, *, bias=None, score="sigmoid", n_group=1, topk_group=1, renorm=True,
               scale=1.0):
    """Top-k experts and their weights for given router logits [T, E] (fp32 or
    bf16): (idx [T, k] int32, w [T, k] fp32).  bias [E] fp32 enters the selection
    only; -inf logits take experts out of a row (moe_route_topk)."""
    dev = _cuda(logits, "logits")
    _need(logits.dim() == 2, "logits must be [T, E]")
    dt = _dtype(logits, "logits")
    _need(score in B.SCORE, f"score must be one of {sorted(B.SCORE)}")
    T, E = logits.shape
    if bias is not None:
        _same(dev, bias=bias)
        _need(bias.dtype == _F32 and bias.shape == (E,), "bias must be an fp32 [E] tensor")
        bias = bias.contiguous()
    with _on(dev) as st:
        logits, ld = _rows(logits)
        idx = torch.empty((T, k), dtype=_I32, device=dev)
        w = torch.empty((T, k), dtype=_F32, device=dev)
        B.moe_route_topk(_ptr(logits), dt, ld, _ptr(bias), T, E, k, B.SCORE[score], n_group,
                         topk_group, int(renorm), scale, _ptr(idx), _ptr(w), st)
    return idx, w


def route_topk_backward(logits, idx, w, dw, *, score="sigmoid", renorm=True, scale=1.0):
    """Gradient of the logits from dw [T, k], given route_topk's arguments and
    results: dlogits [T, E] in the logits' type."""
    dev = _cuda(logits, "logits")
    _need(logits.dim() == 2 and idx.dim() == 2, "logits must be [T, E] and idx [T, k]")
    dt = _dtype(logits, "logits")
    _need(score in B.SCORE, f"score must be one of {sorted(B.SCORE)}")
    T, E = logits.shape
    k = idx.shape[1]
    _same(dev, idx=idx, w=w, dw=dw)
    _need(idx.dtype == _I32 and idx.shape[0] == T, "idx must be int32 [T, k]")
    _need(w.dtype == _F32 and w.shape == idx.shape, "w must be fp32 [T, k]")
    _need(dw.dtype == _F32 and dw.shape == idx.shape, "dw must be fp32 [T, k]")
    with _on(dev) as st:
        logits, ld = _rows(logits)
        idx, w, dw = idx.contiguous(), w.contiguous(), dw.contiguous()
        dl = torch.empty((T, E), dtype=logits.dtype, device=dev)
        B.moe_route_topk_backward(_ptr(logits), dt, ld, _ptr(idx), _ptr(w), _ptr(dw), T, E, k,
                                  B.SCORE[score], int(renorm), scale, _ptr(dl), E, st)
    return dl


def route_group(idx, n_experts):
    """The pairs t*k + j of idx [T, k] by expert: (counts [E], offsets [E + 1],
    perm [T*k], pos [T*k]), int32 (moe_route_group)."""
    dev = _cuda(idx, "idx")
    _need(idx.dim() == 2 and idx.dtype == _I32, "idx must be int32 [T, k]")
    T, k = idx.shape
    with _on(dev) as st:
        idx = idx.contiguous()
        counts = torch.empty(n_experts, dtype=_I32, device=dev)
        offsets = torch.empty(n_experts + 1, dtype=_I32, device=dev)
        perm = torch.empty(T * k, dtype=_I32, device=dev)
        pos = torch.empty(T * k, dtype=_I32, device=dev)
        n = B.moe_route_group_workspace(T, k, n_experts)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        B.moe_route_group(_ptr(idx), T, k, n_experts, _ptr(counts), _ptr(offsets), _ptr(perm),
                          _ptr(pos), _ptr(ws), n, st)
    return counts, offsets, perm, pos


# ---------------------------------------------------------------------------
# norms, gate and residual
# ---------------------------------------------------------------------------
def _gate_kind(gate, T, D):
    if gate is None:
        return B.MOE_GATE_NONE
    if gate.dim() == 1 and gate.shape[0] == D:
        return B.MOE_GATE_CHANNEL
    _need(gate.dim() == 2 and gate.shape[0] == T and gate.shape[1] in (1, D),
          "gate must be [D], [T, 1] or [T, D]")
    return B.MOE_GATE_FULL if gate.shape[1] == D and D > 1 else B.MOE_GATE_TOKEN


def _norm_args(shape, dtype, dev, y, r, post_weight, gate, residual_scale, pre_weight, eps):
    """The fields that forward and backward share; the tensors that its
    pointers come from are kept in the second result."""
    T, D = shape
    a = B.moe_norm_args(T=T, D=D, dtype=_CODE[dtype], residual_scale=residual_scale, eps=eps)
    a.gate_kind = _gate_kind(gate, T, D)
    for n, w in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        _need(w is None or (w.dtype == dtype and w.shape == (D,)), f"{n} must be [D] in x's type")
    _need(gate is None or gate.dtype == dtype, "gate must have x's type")
    _same(dev, y=y, post_weight=post_weight, pre_weight=pre_weight, gate=gate)
    _need(y.shape == shape and y.dtype == dtype, "y must have x's shape and type")
    y, a.ldy = _rows16(y)
    keep = [y]
    a.y = y.data_ptr()
    if r is not None:
        r, a.ldr = _rows16(r)
        a.r = r.data_ptr()
        keep.append(r)
    for n, w in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if w is not None:
            w = _vec16(w)
            setattr(a, n, w.data_ptr())
            keep.append(w)
    if gate is not None:
        if a.gate_kind == B.MOE_GATE_FULL:
            gate, a.ldg = _rows16(gate)
        elif a.gate_kind == B.MOE_GATE_TOKEN:
            gate = gate.contiguous()
            a.ldg = 1
        else:
            gate = _vec16(gate)
        a.gate = gate.data_ptr()
        keep.append(gate)
    return a, keep


def norm_residual(x, y, *, post_weight=None, gate=None, residual_scale=1.0, pre_weight=None,
                  eps=1e-5, stats=False):
    """r = residual_scale * x + gate * norm(y; post_weight) and, with pre_weight,
    h = norm(r; pre_weight), x and y [T, D] fp32 or bf16.  gate: None, [D],
    [T, 1] or [T, D].  stats keeps the reciprocal norms, which
    norm_residual_backward reads."""
    dev = _cuda(x, "x")
    _need(x.dim() == 2, "x must be [T, D]")
    _dtype(x, "x")
    T, D = x.shape
    with _on(dev) as st:
        a, keep = _norm_args(x.shape, x.dtype, dev, y, None, post_weight, gate, residual_scale,
                             pre_weight, eps)
        x, a.ldx = _rows16(x)
        a.x = x.data_ptr()
        r = torch.empty((T, D), dtype=x.dtype, device=dev)
        a.r, a.ldr = r.data_ptr(), D
        h = ry = rr = None
        if pre_weight is not None:
            h = torch.empty((T, D), dtype=x.dtype, device=dev)
            a.h, a.ldh = h.data_ptr(), D
        if stats and post_weight is not None:
            ry = torch.empty(T, dtype=_F32, device=dev)
            a.rstd_y = ry.data_ptr()
        if stats and pre_weight is not None:
            rr = torch.empty(T, dtype=_F32, device=dev)
            a.rstd_r = rr.data_ptr()
        B.moe_norm_residual(a, st)
    return NormForward(r, h, ry, rr)


def norm_residual_backward(dr, dh, y, forward, *, post_weight=None, gate=None, residual_scale=1.0,
                           pre_weight=None):
    """Gradients of norm_residual(.., stats=True), whose result is `forward`,
    from dr (None for zero) and dh (with pre_weight): dx, dy in their type,
    dpost_weight, dpre_weight fp32 [D], dgate fp32 [D] / [T, 1] or [T, D] in the
    gate's type."""
    r = forward.r
    dev = _cuda(r, "forward.r")
    T, D = r.shape
    _need((dh is not None) == (pre_weight is not None), "dh goes with pre_weight")
    _need(post_weight is None or forward.rstd_y is not None, "forward ran without stats")
    _need(pre_weight is None or forward.rstd_r is not None, "forward ran without stats")
    _same(dev, dr=dr, dh=dh)
    with _on(dev) as st:
        a, keep = _norm_args(r.shape, r.dtype, dev, y, r, post_weight, gate, residual_scale,
                             pre_weight, 1.0)
        for n, t in (("dr", dr), ("dh", dh)):
            if t is not None:
                _need(t.shape == r.shape and t.dtype == r.dtype, f"{n} must have x's shape and type")
                t, ld = _rows16(t)
                setattr(a, n, t.data_ptr())
                setattr(a, "ld" + n, ld)
                keep.append(t)
        a.rstd_y, a.rstd_r = _ptr(forward.rstd_y), _ptr(forward.rstd_r)
        dx = torch.empty((T, D), dtype=r.dtype, device=dev)
        dy = torch.empty((T, D), dtype=r.dtype, device=dev)
        a.dx, a.lddx, a.dy, a.lddy = dx.data_ptr(), D, dy.data_ptr(), D
        dpost = dpre = dgate = None
        if post_weight is not None:
            dpost = torch.empty(D, dtype=_F32, device=dev)
            a.dpost_weight = dpost.data_ptr()
        if pre_weight is not None:
            dpre = torch.empty(D, dtype=_F32, device=dev)
            a.dpre_weight = dpre.data_ptr()
        if gate is not None:
            full = a.gate_kind == B.MOE_GATE_FULL
            dgate = torch.empty(gate.shape, dtype=r.dtype if full else _F32, device=dev)
            a.dgate, a.lddg = dgate.data_ptr(), D
        n = B.moe_norm_residual_workspace(T, D)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        B.moe_norm_residual_backward(a, _ptr(ws), n, st)
    return NormBackward(dx, dy, dpost, dpre, dgate)


# ---------------------------------------------------------------------------
# 8-bit products
# ---------------------------------------------------------------------------
def quantize_fp8(x, *, perm=None, k=1, relu2=False, transpose=False):
    """x [M, K] (fp32 or bf16) as E4M3 codes with a scale for each 128 of a row.
    perm [R] int32: row r of the result is row perm[r] // k of x (zeros for a
    negative entry).  relu2: of max(x, 0)^2.  transpose: of x's transpose, so
    codes [K, M]."""
    dev = _cuda(x, "x")
    _need(x.dim() == 2, "x must be [M, K]")
    dt = _dtype(x, "x")
    M, K = x.shape
    _need(not transpose or (perm is None and not relu2), "transpose takes neither perm nor relu2")
    with _on(dev) as st:
        x, ld = _rows(x)
        if transpose:
            codes = torch.empty((K, _up16(M)), dtype=_F8, device=dev)
            scales = torch.empty((_blocks(M), K), dtype=_F32, device=dev)
            B.moe_quantize_fp8_t(_ptr(x), dt, M, K, ld, _ptr(codes), codes.shape[1], _ptr(scales),
                                 K, st)
            return Fp8(codes[:, :M], scales)
        R = M
        if perm is not None:
            _same(dev, perm=perm)
            _need(perm.dim() == 1 and perm.dtype == _I32, "perm must be int32 [R]")
            perm = perm.contiguous()
            R = perm.shape[0]
        codes = torch.empty((R, _up16(K)), dtype=_F8, device=dev)
        scales = torch.empty((_blocks(K), R), dtype=_F32, device=dev)
        B.moe_quantize_fp8(_ptr(x), dt, M, K, ld, _ptr(perm), R, k, int(relu2), _ptr(codes),
                           codes.shape[1], _ptr(scales), R, st)
    return Fp8(codes[:, :K], scales)


def quantize_fp8_weight(w, *, transposed=False):
    """w [N, K] or [E, N, K] with a scale for each 128 x 128 block; with
    `transposed` also the transpose (of each matrix): (Fp8, Fp8)."""
    dev = _cuda(w, "w")
    _need(w.dim() in (2, 3), "w must be [N, K] or [E, N, K]")
    dt = _dtype(w, "w")
    lead = tuple(w.shape[:-2])
    N, K = w.shape[-2:]
    with _on(dev) as st:
        w = w.contiguous()
        codes = torch.empty(lead + (N, _up16(K)), dtype=_F8, device=dev)
        scales = torch.empty(lead + (_blocks(N), _blocks(K)), dtype=_F32, device=dev)
        ct = sc = None
        if transposed:
            ct = torch.empty(lead + (K, _up16(N)), dtype=_F8, device=dev)
            sc = torch.empty(lead + (_blocks(K), _blocks(N)), dtype=_F32, device=dev)
        B.moe_quantize_fp8_weight(_ptr(w), dt, lead[0] if lead else 1, N, K, K, _ptr(codes),
                                  _up16(K), _ptr(scales), _ptr(ct), _up16(N), _ptr(sc), st)
    q = Fp8(codes[..., :K], scales)
    return (q, Fp8(ct[..., :N], sc)) if transposed else q


def _codes(t, what):
    """Codes whose rows are as the library reads them, and the row stride."""
    _need(t.dtype in (_F8, torch.uint8), f"{what}.codes must be float8_e4m3fn or uint8")
    ld, N = t.stride(-2), t.shape[-2]
    ok = (t.stride(-1) == 1 or t.shape[-1] == 1) and ld % 16 == 0 and ld >= t.shape[-1] and \
        t.data_ptr() % 16 == 0 and (t.dim() == 2 or t.stride(0) == N * ld or t.shape[0] == 1)
    if not ok:
        p = torch.empty(t.shape[:-1] + (_up16(t.shape[-1]),), dtype=t.dtype, device=t.device)
        p[..., :t.shape[-1]] = t
        t, ld = p, p.shape[-1]
    return t, ld


def gemm_fp8(a, b, *, offsets=None, out_dtype="bf16", out=None):
    """out[m, n] = sum_k A[m, k] B[n, k] for a: Fp8 rows [M, K] and b: Fp8
    weights [N, K], or rows [N, K] (the weight gradient).  With offsets [E + 1]
    int32 and b [E, N, K], rows [offsets[e], offsets[e + 1]) take b's matrix e;
    rows of `out` in no group keep their contents."""
    dev = _cuda(a.codes, "a.codes")
    _need(a.codes.dim() == 2, "a.codes must be [M, K]")
    M, K = a.codes.shape
    KB = _blocks(K)
    _same(dev, a_scales=a.scales, b_codes=b.codes, b_scales=b.scales, offsets=offsets, out=out)
    _need(a.scales.dtype == _F32 and a.scales.shape == (KB, M), "a.scales must be fp32 [ceil(K/128), M]")
    grouped = offsets is not None
    _need(b.codes.dim() == (3 if grouped else 2) and b.codes.shape[-1] == K,
          "b.codes must be [N, K], or [E, N, K] with offsets")
    N = b.codes.shape[-2]
    lead = tuple(b.codes.shape[:-2])
    _need(b.scales.dtype == _F32, "b.scales must be fp32")
    # [NB, KB] and [KB, N] agree only at N = 1, K <= 128, where both are the one scale
    weights = tuple(b.scales.shape) == lead + (_blocks(N), KB)
    _need(weights or (not grouped and tuple(b.scales.shape) == (KB, N)),
          "b.scales must be [.., ceil(N/128), ceil(K/128)], or [ceil(K/128), N]")
    if out is None:
        _need(out_dtype in _OUT, f"out_dtype must be one of {sorted(_OUT)}")
    else:
        _need(out.shape == (M, N) and out.dtype in _CODE and (out.stride(1) == 1 or N == 1)
              and (out.stride(0) >= N or M <= 1), "out must be [M, N], rows contiguous")
    with _on(dev) as st:
        if out is None:
            out = torch.empty((M, N), dtype=_OUT[out_dtype], device=dev)
        ac, lda = _codes(a.codes, "a")
        bc, ldb = _codes(b.codes, "b")
        a_scales, lds = _rows(a.scales)
        g = B.moe_fp8_gemm(M=M, N=N, K=K, a=_ptr(ac), lda=lda, a_scales=_ptr(a_scales),
                           lda_scales=lds, b=_ptr(bc), ldb=ldb, out=_ptr(out),
                           ldo=max(out.stride(0), N), out_dtype=_CODE[out.dtype])
        if weights:
            b_scales = b.scales.contiguous()
        else:
            b_scales, g.ldb_scales = _rows(b.scales)
        g.b_scales = _ptr(b_scales)
        if grouped:
            _need(offsets.dtype == _I32 and offsets.shape == (lead[0] + 1,),
                  "offsets must be int32 [E + 1]")
            offsets = offsets.contiguous()
            g.offsets, g.n_groups = _ptr(offsets), lead[0]
        B.moe_gemm_fp8(g, st)
    return out
