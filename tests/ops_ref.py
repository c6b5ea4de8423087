"""Plain 64-bit forms of the stand-alone operators, for their tests (CPU)."""
import numpy as np
import torch

F64 = torch.float64


def scores64(logits, score):
    """(s [T, E] in 64 bits, live): a -inf or NaN logit has no part."""
    l = logits.detach().cpu().to(F64).numpy()
    live = l > -np.inf
    out = np.zeros_like(l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            out[live] = 1.0 / (1.0 + np.exp(-l[live]))
        return out, live
    for t in range(l.shape[0]):
        x = l[t][live[t]]
        if x.size:
            m = x.max()
            e = np.where(x == m, 1.0, np.exp(np.where(x == m, 0.0, x - m)))
            out[t][live[t]] = e / e.sum()
    return out, live


def route(logits, k, bias=None, score="sigmoid", n_group=1, topk_group=1, renorm=True, scale=1.0):
    """(idx [T, k], w [T, k] 64-bit, chosen [T, k]) row by row, by sorting."""
    s, live = scores64(logits, score)
    T, E = s.shape
    b = np.zeros(E, np.float32) if bias is None else bias.detach().cpu().numpy()
    idx, w, chosen = np.zeros((T, k), np.int32), np.zeros((T, k)), np.zeros((T, k), bool)
    for t in range(T):
        with np.errstate(invalid="ignore"):
            c = s[t].astype(np.float32) + b
        ok = live[t] & (c > -np.inf)
        c = np.where(ok, c, np.float32(-np.inf))
        if n_group > 1:
            G = E // n_group
            top2 = [np.sort(c[g * G:(g + 1) * G])[::-1][:2] for g in range(n_group)]
            gs = [np.float32(a) + np.float32(d) for a, d in top2]
            keep = sorted(range(n_group), key=lambda g: (-gs[g], g))[:topk_group]
            for g in range(n_group):
                if g not in keep:
                    c[g * G:(g + 1) * G] = -np.inf
        order = sorted(range(E), key=lambda e: (-c[e], e))[:k]
        idx[t] = order
        chosen[t] = c[order] > -np.inf
        p = np.where(chosen[t], s[t][order].astype(np.float32).astype(np.float64), 0.0)
        w[t] = p / (p.sum() + 1e-20) * scale if renorm else p * scale
    return idx, w, chosen


def route_weights(logits, idx, chosen, score, renorm, scale):
    """The weights as a differentiable 64-bit function of the logits, for fixed
    indices: what the gradient belongs to."""
    l = logits
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    p = torch.gather(s, 1, idx.long()) * chosen
    return p / (p.sum(1, keepdim=True) + 1e-20) * scale if renorm else p * scale


def route_backward(logits, idx, chosen, dw, score, renorm, scale):
    """dlogits in 64 bits by the formulas, masked logits included."""
    s, _ = scores64(logits, score)
    T, E = s.shape
    i = idx.cpu().numpy()
    rows = np.arange(T)[:, None]
    p = np.where(chosen, s[rows, i], 0.0)
    u = np.where(chosen, dw.detach().cpu().to(F64).numpy() * scale, 0.0)
    if renorm:
        S = p.sum(1, keepdims=True) + 1e-20
        ds = (u - (u * (p / S)).sum(1, keepdims=True)) / S
    else:
        ds = u
    full = np.zeros((T, E))
    full[rows, i] = ds
    if score == "sigmoid":
        return full * s * (1.0 - s)
    return s * (full - (full * s).sum(1, keepdims=True))


def group(idx, E):
    flat = np.asarray(idx).reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = [p for e in range(E) for p in np.nonzero(flat == e)[0]]
    counts = np.bincount(flat[ok], minlength=E)
    perm = np.full(flat.size, -1)
    perm[:len(order)] = order
    pos = np.full(flat.size, -1)
    pos[order] = np.arange(len(order))
    return counts, np.concatenate([[0], np.cumsum(counts)]), perm, pos


def rms(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def norm_r(x, y, post_weight, gate, alpha, eps):
    """The residual in 64 bits, before it is rounded."""
    x, y = x.cpu().to(F64), y.cpu().to(F64)
    n = y if post_weight is None else y * rms(y, eps) * post_weight.cpu().to(F64)
    return alpha * x + (n if gate is None else gate.cpu().to(F64) * n)


def norm_h(r, pre_weight, eps):
    r = r.cpu().to(F64)
    return r * rms(r, eps) * pre_weight.cpu().to(F64)


def e4m3_grid():
    """The finite non-negative values of E4M3, ascending."""
    v = [m / 8 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:-1])            # the last code is NaN


def e4m3_round(t):
    """Nearest E4M3 value of 64-bit t, ties to the even code, saturating."""
    g = e4m3_grid()
    a = np.minimum(np.abs(t), g[-1])
    hi = np.clip(np.searchsorted(g, a), 1, len(g) - 1)
    lo = hi - 1
    dl, dh = a - g[lo], g[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.copysign(g[pick], t)


def quantize(x, block_rows=1):
    """(codes' values, scales [row blocks, K blocks]) of x [R, K] in blocks of
    block_rows x 128; scale, factor and product are single fp32 operations."""
    x = x.detach().cpu().float().numpy()
    R, K = x.shape
    RB, KB = -(-R // block_rows), -(-K // 128)
    codes, scales = np.zeros((R, K)), np.zeros((RB, KB), np.float32)
    for i in range(RB):
        for j in range(KB):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            m = np.maximum(np.abs(x[at]).max(), np.float32(2.0 ** -100)).astype(np.float32)
            scales[i, j] = m / np.float32(448)
            codes[at] = e4m3_round((x[at] * (np.float32(448) / m)).astype(np.float64))
    return codes, scales


def values(codes, scales, block_rows=1):
    """codes * scales in 64 bits; scales [row blocks, K blocks]."""
    R, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), block_rows, 0)[:R], 128, 1)[:, :K]
    return codes * s
