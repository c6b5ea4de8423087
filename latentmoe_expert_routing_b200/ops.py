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
MoeError; what kernels find wrong on the device (an expert out of range, a wait
that ran out) is kept until sync() raises it.  What the C calls expect and
promise stands in include/latentmoe.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B

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


# The calls are short next to a decoding step, so what surrounds them is kept
# short too: the current stream's raw handle, sizes as numbers (torch.empty takes
# them faster than a tuple), checks in line.
_device = torch._C._cuda_getDevice
_set_device = torch.cuda.set_device
_stream = torch._C._cuda_getCurrentRawStream
_empty = torch.empty
_Tensor = torch.Tensor
_F32, _BF16, _I32, _F8, _U8 = (torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn,
                               torch.uint8)
_CODE = {_F32: B.MOE_FP32, _BF16: B.MOE_BF16}
_OUT = {"fp32": _F32, "bf16": _BF16}


class _on:
    """Makes a device current for a call; entered only when it is not."""

    def __init__(self, dev):
        self.dev = dev

    def __enter__(self):
        self.old = _device()
        _set_device(self.dev)

    def __exit__(self, *exc):
        _set_device(self.old)


def _bad(what):
    raise ValueError(what)


def _input(t, what, dims=2):
    """The device index and dtype code of a cuda fp32 / bf16 matrix."""
    if not (isinstance(t, _Tensor) and t.is_cuda):
        _bad(f"{what} must be a cuda tensor")
    if t.dim() != dims:
        _bad(f"{what} must have {dims} dimensions")
    dt = _CODE.get(t.dtype)
    if dt is None:
        _bad(f"{what} must be float32 or bfloat16")
    return t.get_device(), dt


def _like(t, what, dev, dtype, shape):
    if not isinstance(t, _Tensor) or t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        _bad(f"{what} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")


def _rows(t):
    """t [R, C] with contiguous rows, and their stride; a copy where t's are not."""
    R, C = t.shape
    sr, sc = t.stride()
    if sc != 1 and C != 1 or sr < C and R > 1:
        return t.contiguous(), C
    return t, sr if sr > C else C


def _rows16(t):
    """The same, each row starting on 16 bytes."""
    t, ld = _rows(t)
    if t.data_ptr() & 15 or ld * t.element_size() & 15:
        t = t.clone(memory_format=torch.contiguous_format)
        ld = t.shape[1]
    return t, ld


def _vec16(t):
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _up16(n):
    return (n + 15) // 16 * 16


def _blocks(n):
    return (n + 127) // 128


def sync(device=None):
    """Waits for the current stream of `device` (the current one), then raises
    MoeError for what the kernels of earlier calls found wrong on that device, and
    clears it (moe_sync without a handle)."""
    here = _device()
    dev = device if isinstance(device, int) else None if device is None else torch.device(device).index
    if dev is not None and dev != here:
        with _on(dev):
            return sync()
    B.moe_sync(None, _stream(here))


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def route_topk(logits, k, *, bias=None, score="sigmoid", n_group=1, topk_group=1, renorm=True,
               scale=1.0):
    """Top-k experts and their weights for given router logits [T, E] (fp32 or
    bf16): (idx [T, k] int32, w [T, k] fp32).  bias [E] fp32 enters the selection
    only; -inf logits take experts out of a row (moe_route_topk).  w is detached
    from logits: route_topk_backward is its gradient."""
    dev, dt = _input(logits, "logits")
    if score not in B.SCORE:
        _bad(f"score must be one of {sorted(B.SCORE)}")
    if k < 0:
        _bad("k must not be negative")
    if dev != _device():
        with _on(dev):
            return route_topk(logits, k, bias=bias, score=score, n_group=n_group,
                              topk_group=topk_group, renorm=renorm, scale=scale)
    T, E = logits.shape
    if bias is not None:
        _like(bias, "bias", dev, _F32, (E,))
        bias = bias.contiguous()
    logits, ld = _rows(logits)
    idx = _empty(T, k, dtype=_I32, device=logits.device)
    w = _empty(T, k, dtype=_F32, device=logits.device)
    B.moe_route_topk(logits.data_ptr(), dt, ld, None if bias is None else bias.data_ptr(), T, E, k,
                     B.SCORE[score], n_group, topk_group, 1 if renorm else 0, scale,
                     idx.data_ptr(), w.data_ptr(), _stream(dev))
    return idx, w


def route_topk_backward(logits, idx, w, dw, *, score="sigmoid", renorm=True, scale=1.0):
    """Gradient of the logits from dw [T, k], given route_topk's arguments and
    results: dlogits [T, E] in the logits' type, detached."""
    dev, dt = _input(logits, "logits")
    if score not in B.SCORE:
        _bad(f"score must be one of {sorted(B.SCORE)}")
    if dev != _device():
        with _on(dev):
            return route_topk_backward(logits, idx, w, dw, score=score, renorm=renorm, scale=scale)
    T, E = logits.shape
    if not isinstance(idx, _Tensor) or idx.dim() != 2:
        _bad("idx must be [T, k]")
    k = idx.shape[1]
    _like(idx, "idx", dev, _I32, (T, k))
    _like(w, "w", dev, _F32, (T, k))
    _like(dw, "dw", dev, _F32, (T, k))
    logits, ld = _rows(logits)
    idx, w, dw = idx.contiguous(), w.contiguous(), dw.contiguous()
    dl = _empty(T, E, dtype=logits.dtype, device=logits.device)
    B.moe_route_topk_backward(logits.data_ptr(), dt, ld, idx.data_ptr(), w.data_ptr(),
                              dw.data_ptr(), T, E, k, B.SCORE[score], 1 if renorm else 0, scale,
                              dl.data_ptr(), E, _stream(dev))
    return dl


def route_group(idx, n_experts):
    """The pairs t*k + j of idx [T, k] by expert: (counts [E], offsets [E + 1],
    perm [T*k], pos [T*k]), int32, views of one buffer (moe_route_group)."""
    if not (isinstance(idx, _Tensor) and idx.is_cuda):
        _bad("idx must be a cuda tensor")
    if idx.dim() != 2 or idx.dtype != _I32:
        _bad("idx must be int32 [T, k]")
    if n_experts < 0:
        _bad("n_experts must not be negative")
    dev = idx.get_device()
    if dev != _device():
        with _on(dev):
            return route_group(idx, n_experts)
    T, k = idx.shape
    idx = idx.contiguous()
    E, P = n_experts, T * k
    need = B.moe_route_group_workspace(T, k, E)
    ws = (need + 15) // 16 * 4                    # the workspace lies in front
    buf = _empty(max(0, ws + 2 * E + 1 + 2 * P), dtype=_I32, device=idx.device)
    at = buf.data_ptr()
    counts = at + 4 * ws
    B.moe_route_group(idx.data_ptr(), T, k, E, counts, counts + 4 * E, counts + 4 * (2 * E + 1),
                      counts + 4 * (2 * E + 1 + P), at, need, _stream(dev))
    v = buf.as_strided
    return (v((E,), (1,), ws), v((E + 1,), (1,), ws + E), v((P,), (1,), ws + 2 * E + 1),
            v((P,), (1,), ws + 2 * E + 1 + P))


# ---------------------------------------------------------------------------
# norms, gate and residual
# ---------------------------------------------------------------------------
def _gate_kind(gate, T, D):
    if gate is None:
        return B.MOE_GATE_NONE
    if not isinstance(gate, _Tensor):
        _bad("gate must be a tensor")
    if gate.shape == (D,):
        return B.MOE_GATE_CHANNEL
    if gate.shape == (T, D) and D > 1:
        return B.MOE_GATE_FULL
    if gate.shape != (T, 1):
        _bad("gate must be [D], [T, 1] or [T, D]")
    return B.MOE_GATE_TOKEN


def _norm_inputs(T, D, r, y, post_weight, gate, pre_weight):
    """(kind, y, ldy, post_weight, pre_weight, gate, ldg) as the library reads
    them: checked against r's shape, type and device, copied where unaligned."""
    dev, dtype = r.get_device(), r.dtype
    if not isinstance(y, _Tensor) or y.shape != r.shape or y.dtype != dtype or y.get_device() != dev:
        _bad("y must have x's shape, type and device")
    y, ldy = _rows16(y)
    if post_weight is not None:
        _like(post_weight, "post_weight", dev, dtype, (D,))
        post_weight = _vec16(post_weight)
    if pre_weight is not None:
        _like(pre_weight, "pre_weight", dev, dtype, (D,))
        pre_weight = _vec16(pre_weight)
    kind, ldg = _gate_kind(gate, T, D), 0
    if kind:
        if gate.dtype != dtype or gate.get_device() != dev:
            _bad("gate must have x's type and device")
        if kind == B.MOE_GATE_FULL:
            gate, ldg = _rows16(gate)
        elif kind == B.MOE_GATE_TOKEN:
            gate, ldg = gate.contiguous(), 1
        else:
            gate = _vec16(gate)
    return kind, y, ldy, post_weight, pre_weight, gate, ldg


def _at(t):
    return None if t is None else t.data_ptr()


def norm_residual(x, y, *, post_weight=None, gate=None, residual_scale=1.0, pre_weight=None,
                  eps=1e-5, stats=False):
    """r = residual_scale * x + gate * norm(y; post_weight) and, with pre_weight,
    h = norm(r; pre_weight), x and y [T, D] fp32 or bf16.  gate: None, [D],
    [T, 1] or [T, D].  stats keeps the reciprocal norms, which
    norm_residual_backward, the gradient, reads: the results are detached."""
    dev, dt = _input(x, "x")
    if dev != _device():
        with _on(dev):
            return norm_residual(x, y, post_weight=post_weight, gate=gate,
                                 residual_scale=residual_scale, pre_weight=pre_weight, eps=eps,
                                 stats=stats)
    T, D = x.shape
    where, dtype = x.device, x.dtype
    kind, y, ldy, post, pre, gate, ldg = _norm_inputs(T, D, x, y, post_weight, gate, pre_weight)
    x, ldx = _rows16(x)
    r = _empty(T, D, dtype=dtype, device=where)
    h = None if pre is None else _empty(T, D, dtype=dtype, device=where)
    ry = _empty(T, dtype=_F32, device=where) if stats and post is not None else None
    rr = _empty(T, dtype=_F32, device=where) if stats and pre is not None else None
    B.moe_norm_residual(B.moe_norm_args(
        T, D, dt, kind, residual_scale, eps, x.data_ptr(), ldx, y.data_ptr(), ldy, _at(post),
        _at(pre), _at(gate), ldg, r.data_ptr(), D, _at(h), D, _at(ry), _at(rr)), _stream(dev))
    return NormForward(r, h, ry, rr)


def norm_residual_backward(dr, dh, y, forward, *, post_weight=None, gate=None, residual_scale=1.0,
                           pre_weight=None):
    """Gradients of norm_residual(.., stats=True), whose result is `forward`,
    from dr (None for zero) and dh (with pre_weight): dx, dy in their type,
    dpost_weight, dpre_weight fp32 [D], dgate fp32 [D] / [T, 1] or [T, D] in the
    gate's type, all detached."""
    try:
        r, _, ry, rr = forward
    except (TypeError, ValueError):
        _bad("forward must be what norm_residual returned")
    dev, dt = _input(r, "forward.r")
    if (dh is not None) != (pre_weight is not None):
        _bad("dh goes with pre_weight")
    if post_weight is not None and ry is None or pre_weight is not None and rr is None:
        _bad("forward ran without stats")
    if dev != _device():
        with _on(dev):
            return norm_residual_backward(dr, dh, y, forward, post_weight=post_weight, gate=gate,
                                          residual_scale=residual_scale, pre_weight=pre_weight)
    T, D = r.shape
    where, dtype = r.device, r.dtype
    shape = getattr(gate, "shape", None)
    kind, y, ldy, post, pre, gate, ldg = _norm_inputs(T, D, r, y, post_weight, gate, pre_weight)
    r, ldr = _rows16(r)
    lddr = lddh = 0
    if dr is not None:
        _like(dr, "dr", dev, dtype, (T, D))
        dr, lddr = _rows16(dr)
    if dh is not None:
        _like(dh, "dh", dev, dtype, (T, D))
        dh, lddh = _rows16(dh)
    if post is not None:
        _like(ry, "forward.rstd_y", dev, _F32, (T,))
    if pre is not None:
        _like(rr, "forward.rstd_r", dev, _F32, (T,))
    dx = _empty(T, D, dtype=dtype, device=where)
    dy = _empty(T, D, dtype=dtype, device=where)
    # the column sums apart from the workspace, which would live as long as they
    need = B.moe_norm_residual_workspace(T, D)
    work = _empty(need, dtype=_U8, device=where)
    sums = _empty(3 * D, dtype=_F32, device=where)
    at, v = sums.data_ptr(), sums.as_strided
    dpost = None if post is None else v((D,), (1,), 0)
    dpre = None if pre is None else v((D,), (1,), D)
    dgate = at_gate = None
    if kind == B.MOE_GATE_CHANNEL:
        dgate, at_gate = v((D,), (1,), 2 * D), at + 8 * D
    elif kind:
        dgate = _empty(*shape, dtype=dtype if kind == B.MOE_GATE_FULL else _F32, device=where)
        at_gate = dgate.data_ptr()
    B.moe_norm_residual_backward(B.moe_norm_args(
        T, D, dt, kind, residual_scale, 1.0, None, 0, y.data_ptr(), ldy, _at(post), _at(pre),
        _at(gate), ldg, r.data_ptr(), ldr, None, 0, _at(ry), _at(rr), _at(dr), lddr, _at(dh), lddh,
        dx.data_ptr(), D, dy.data_ptr(), D, None if post is None else at,
        None if pre is None else at + 4 * D, at_gate, D), work.data_ptr(), need, _stream(dev))
    return NormBackward(dx, dy, dpost, dpre, dgate)


# ---------------------------------------------------------------------------
# 8-bit products
# ---------------------------------------------------------------------------
def quantize_fp8(x, *, perm=None, k=1, relu2=False, transpose=False):
    """x [M, K] (fp32 or bf16) as E4M3 codes with a scale for each 128 of a row.
    perm [R] int32: row r of the result is row perm[r] // k of x (zeros for an
    entry that names no row).  relu2: of max(x, 0)^2.  transpose: of x's
    transpose, so codes [K, M].  The codes carry no gradient."""
    dev, dt = _input(x, "x")
    if dev != _device():
        with _on(dev):
            return quantize_fp8(x, perm=perm, k=k, relu2=relu2, transpose=transpose)
    M, K = x.shape
    where = x.device
    x, ld = _rows(x)
    if transpose:
        if perm is not None or relu2:
            _bad("transpose takes neither perm nor relu2")
        ldc = _up16(M)
        codes = _empty(K, ldc, dtype=_F8, device=where)
        scales = _empty(_blocks(M), K, dtype=_F32, device=where)
        B.moe_quantize_fp8_t(x.data_ptr(), dt, M, K, ld, codes.data_ptr(), ldc, scales.data_ptr(),
                             K, _stream(dev))
        return Fp8(codes if ldc == M else codes[:, :M], scales)
    R, at = M, None
    if perm is not None:
        if not isinstance(perm, _Tensor) or perm.dim() != 1 or perm.dtype != _I32 or perm.get_device() != dev:
            _bad("perm must be int32 [R] on x's device")
        perm = perm.contiguous()
        R, at = perm.shape[0], perm.data_ptr()
    ldc = _up16(K)
    codes = _empty(R, ldc, dtype=_F8, device=where)
    scales = _empty(_blocks(K), R, dtype=_F32, device=where)
    B.moe_quantize_fp8(x.data_ptr(), dt, M, K, ld, at, R, k, 1 if relu2 else 0, codes.data_ptr(),
                       ldc, scales.data_ptr(), R, _stream(dev))
    return Fp8(codes if ldc == K else codes[:, :K], scales)


def quantize_fp8_weight(w, *, transposed=False):
    """w [N, K] or [E, N, K] with a scale for each 128 x 128 block; with
    `transposed` also the transpose (of each matrix): (Fp8, Fp8).  The codes carry
    no gradient."""
    dev, dt = _input(w, "w", 3 if isinstance(w, _Tensor) and w.dim() == 3 else 2)
    if dev != _device():
        with _on(dev):
            return quantize_fp8_weight(w, transposed=transposed)
    lead = tuple(w.shape[:-2])
    N, K = w.shape[-2:]
    where = w.device
    w = w.contiguous()
    codes = _empty(*lead, N, _up16(K), dtype=_F8, device=where)
    scales = _empty(*lead, _blocks(N), _blocks(K), dtype=_F32, device=where)
    ct = sc = None
    if transposed:
        ct = _empty(*lead, K, _up16(N), dtype=_F8, device=where)
        sc = _empty(*lead, _blocks(K), _blocks(N), dtype=_F32, device=where)
    B.moe_quantize_fp8_weight(w.data_ptr(), dt, lead[0] if lead else 1, N, K, K, codes.data_ptr(),
                              _up16(K), scales.data_ptr(), ct.data_ptr() if transposed else None,
                              _up16(N), sc.data_ptr() if transposed else None, _stream(dev))
    q = Fp8(codes[..., :K], scales)
    return (q, Fp8(ct[..., :N], sc)) if transposed else q


def _codes(t, what):
    """Codes whose rows are as the library reads them, and the row stride."""
    if t.dtype != _F8 and t.dtype != _U8:
        _bad(f"{what}.codes must be float8_e4m3fn or uint8")
    st, N, K = t.stride(), t.shape[-2], t.shape[-1]
    ld = st[-2] if N > 1 else max(_up16(K), st[-2])
    if (st[-1] == 1 or K == 1) and not ld & 15 and ld >= K and not t.data_ptr() & 15 and \
            (len(st) == 2 or st[0] == N * ld or t.shape[0] == 1):
        return t, ld
    p = _empty(*t.shape[:-1], _up16(K), dtype=t.dtype, device=t.device)
    p[..., :K] = t
    return p, p.shape[-1]


def gemm_fp8(a, b, *, offsets=None, out_dtype="bf16", out=None):
    """out[m, n] = sum_k A[m, k] B[n, k] for a: Fp8 rows [M, K] and b: Fp8
    weights [N, K], or rows [N, K] (the weight gradient).  With offsets [E + 1]
    int32 and b [E, N, K], rows [offsets[e], offsets[e + 1]) take b's matrix e;
    rows of `out` in no group keep their contents.  Without offsets K may be 0 (the
    weight gradient of a batch without rows): zeros.  The result is detached: its
    gradients are two more products (dx = dy times W's transpose, dW = dy's
    transpose times x's)."""
    try:
        ac, bc, a_scales, b_scales = a.codes, b.codes, a.scales, b.scales
    except AttributeError:
        _bad("a and b must be Fp8")
    if not (isinstance(ac, _Tensor) and ac.is_cuda):
        _bad("a.codes must be a cuda tensor")
    dev = ac.get_device()
    if dev != _device():
        with _on(dev):
            return gemm_fp8(a, b, offsets=offsets, out_dtype=out_dtype, out=out)
    if not isinstance(bc, _Tensor) or ac.dim() != 2 or bc.dim() != (2 if offsets is None else 3):
        _bad("a.codes must be [M, K] and b.codes [N, K], or [E, N, K] with offsets")
    M, K = ac.shape
    N = bc.shape[-2]
    if bc.shape[-1] != K or bc.get_device() != dev:
        _bad("b.codes must have a.codes' K and device")
    KB = _blocks(K)
    _like(a_scales, "a.scales", dev, _F32, (KB, M))
    if not isinstance(b_scales, _Tensor) or b_scales.dtype != _F32 or b_scales.get_device() != dev:
        _bad("b.scales must be fp32 on a's device")
    # [NB, KB] and [KB, N] agree only at N = 1, K <= 128, where both are the one scale
    weights = b_scales.shape == (*bc.shape[:-2], _blocks(N), KB)
    if not weights and (offsets is not None or b_scales.shape != (KB, N)):
        _bad("b.scales must be [.., ceil(N/128), ceil(K/128)], or [ceil(K/128), N]")
    if out is None:
        dtype = _OUT.get(out_dtype)
        if dtype is None:
            _bad(f"out_dtype must be one of {sorted(_OUT)}")
        out = _empty(M, N, dtype=dtype, device=ac.device)
    elif not isinstance(out, _Tensor) or out.shape != (M, N) or out.dtype not in _CODE or \
            out.get_device() != dev or out.stride(1) != 1 and N != 1 or out.stride(0) < N and M > 1:
        _bad("out must be [M, N], fp32 or bf16, rows contiguous, on a's device")
    if K == 0 and offsets is None:
        return out.zero_()
    ac, lda = _codes(ac, "a")
    bc, ldb = _codes(bc, "b")
    a_scales, lds = _rows(a_scales)
    g = B.moe_fp8_gemm(M, N, K, 0, None, ac.data_ptr(), lda, a_scales.data_ptr(), lds,
                       bc.data_ptr(), ldb, 0, 0, out.data_ptr(), max(out.stride(0), N),
                       _CODE[out.dtype])
    if weights:
        b_scales = b_scales.contiguous()
    else:
        b_scales, g.ldb_scales = _rows(b_scales)
    g.b_scales = b_scales.data_ptr()
    if offsets is not None:
        E = bc.shape[0]
        _like(offsets, "offsets", dev, _I32, (E + 1,))
        offsets = offsets.contiguous()
        g.offsets, g.n_groups = offsets.data_ptr(), E
    B.moe_gemm_fp8(g, _stream(dev))
    return out
