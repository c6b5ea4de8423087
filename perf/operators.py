"""The stand-alone operators around a LatentMoE layer, as a user's program calls
them, beside their plain forms.

  route    top-k routing from given router logits: sigmoid or softmax scores, a
           selection bias, expert groups, renormalised weights; the grouping of
           the chosen (token, expert) pairs by expert; the gradient of the logits
  norm     what stands between two blocks of a residual stream: the norm after a
           block, its gate, the scaled residual add and the next block's norm,
           and their gradients
  linear   products of 8-bit floating point operands with one scale for each
           block of 128: quantisation, y = x W^T, and the two products of its
           gradient
  experts  the same products for experts whose rows are grouped by expert: up
           projection, squared ReLU, down projection

With `own` false `run` computes them by elementary torch operations; with `own`
true it calls the library.
"""
import math

import numpy as np
import torch

own = False

F8_MAX = 448.0
F8_FLOOR = 2.0 ** -100          # a block's maximum counts as at least this
NORM_EPS = 1e-5
RENORM_EPS = 1e-20


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    route = dict(op="route", dtype="fp32", score="sigmoid", bias=True, groups=1, keep=1, renorm=True,
                 scale=5.0, dead=0, pad=0, grouping=False, backward=False)
    norm = dict(op="norm", dtype="bf16", post=True, gate="channel", pre=True, alpha=1.0, backward=True)
    return [
        # one decoding step of the Ultra layer: 64 tokens, the call's latency
        dict(route, name="route_decode", T=64, E=512, k=22),
        # its prefill: routing and the grouping by expert that the products need
        dict(route, name="route_prefill", T=16384, E=512, k=22, grouping=True),
        # a training step of a softmax router at the Super's 128 experts, bf16 logits,
        # weights not renormalised: every logit gets a gradient
        dict(route, name="route_train", T=8192, E=128, k=8, dtype="bf16", score="softmax", bias=False,
             renorm=False, scale=1.0, backward=True),
        # grouped routing with experts taken out of service and padded rows
        dict(route, name="route_groups", T=2001, E=256, k=8, groups=8, keep=4, scale=2.5, dead=9, pad=17,
             grouping=True, backward=True),
        # between two blocks while decoding: latency
        dict(norm, name="norm_decode", T=64, D=8192, backward=False),
        # between two blocks in training, the layer's width and prefill batch
        dict(norm, name="norm_train", T=8192, D=8192),
        # fp32, an odd width, a gate for every element, a shrunk residual
        dict(norm, name="norm_odd_fp32", T=777, D=2056, dtype="fp32", gate="full", alpha=0.5),
        # the shared expert's up projection: a decoding batch, then a prefill batch
        dict(op="linear", name="linear_decode", M=64, K=8192, N=10240, out="bf16", train=False),
        dict(op="linear", name="linear_prefill", M=8192, K=8192, N=10240, out="bf16", train=False),
        # fc1 in training: the weights quantised anew, the product, both gradients
        dict(op="linear", name="linear_train", M=4096, K=8192, N=2048, out="bf16", train=True),
        # routed experts of the Ultra's sizes on the latent rows: decoding, prefill
        dict(op="experts", name="experts_decode", T=32, E=64, k=22, L=2048, F=5120),
        dict(op="experts", name="experts_prefill", T=2048, E=64, k=22, L=2048, F=5120),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _step(rng, lo, hi, step):
    return max(lo, _spread(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(("route", "route", "norm", "norm", "linear", "linear", "experts"))
    if op == "route":
        groups, keep = rng.choice(((1, 1), (1, 1), (4, 2), (8, 3)))
        E = _spread(rng, 8 if groups == 1 else 32, 512) // groups * groups
        k = rng.randint(2, min(24, E // groups * keep))
        T = _spread(rng, 1, 16384)
        return dict(op=op, T=T, E=E, k=k, dtype=rng.choice(("fp32", "bf16")),
                    score=rng.choice(("sigmoid", "softmax")), bias=rng.random() < 0.6, groups=groups,
                    keep=keep, renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5, 5.0)),
                    dead=rng.choice((0, 0, E // 16)), pad=rng.choice((0, 0, T // 8)),
                    grouping=rng.random() < 0.5, backward=rng.random() < 0.6)
    if op == "norm":
        T = _spread(rng, 1, 8192)
        D = _step(rng, 64, min(16384, 8192 * 8192 // T), 8)
        return dict(op=op, T=T, D=D, dtype=rng.choice(("bf16", "bf16", "fp32")) if T * D <= 1 << 25 else "bf16",
                    post=rng.random() < 0.8, gate=rng.choice(("none", "channel", "token", "full")),
                    pre=rng.random() < 0.8, alpha=rng.choice((1.0, 0.5, 0.70710678)),
                    backward=rng.random() < 0.6)
    if op == "linear":
        train = rng.random() < 0.4
        return dict(op=op, M=_spread(rng, 1, 4096 if train else 8192), K=_step(rng, 128, 8192, 8),
                    N=_step(rng, 64, 2048 if train else 10240, 8), out=rng.choice(("bf16", "fp32")), train=train)
    E = _spread(rng, 2, 64)
    return dict(op=op, T=_spread(rng, 1, 2048), E=E, k=rng.randint(1, min(16, E)),
                L=_step(rng, 128, 2048, 8), F=_step(rng, 128, 5120, 8))


def _up16(n):
    return (n + 15) // 16 * 16


def _blocks(n):
    return (n + 127) // 128


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(*shape, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=g).to(dtype)


def _weights(g, mats, N, K):
    """E4M3 codes [mats, N, K] in rows of whole 16 bytes, and a scale for each
    128 x 128 block: what a checkpoint of this form holds (a maximum-based scale
    uses the whole range of the type)."""
    codes = torch.zeros(mats, N, _up16(K), device="cuda", dtype=torch.float8_e4m3fn)
    codes[:, :, :K] = _normal(g, mats, N, K, std=110.0).clamp_(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
    scales = torch.empty(mats, _blocks(N), _blocks(K), device="cuda").uniform_(0.8, 1.2, generator=g)
    return codes[:, :, :K], scales * (1.0 / (110.0 * math.sqrt(K)))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        c["logits"] = _normal(g, T, E).to(_dt(c["dtype"]))
        if c["dead"]:          # experts out of service: no token may reach them
            c["logits"][:, torch.randperm(E, generator=g, device="cuda")[: c["dead"]]] = -math.inf
        if c["pad"]:           # rows behind the last sequence
            c["logits"][T - c["pad"]:] = -math.inf
        c["b"] = _normal(g, E, std=0.1) if c["bias"] else None
        c["dw"] = _normal(g, T, k) if c["backward"] else None
    elif c["op"] == "norm":
        T, D, dt = c["T"], c["D"], _dt(c["dtype"])
        c["x"], c["y"] = _normal(g, T, D, std=2.0, dtype=dt), _normal(g, T, D, std=0.7, dtype=dt)
        c["post_w"] = (1.0 + _normal(g, D, std=0.1)).to(dt) if c["post"] else None
        c["pre_w"] = (1.0 + _normal(g, D, std=0.1)).to(dt) if c["pre"] else None
        shape = {"none": None, "channel": (D,), "token": (T, 1), "full": (T, D)}[c["gate"]]
        c["g"] = None if shape is None else (0.5 + _normal(g, *shape, std=0.2)).to(dt)
        c["dr"] = _normal(g, T, D, dtype=dt) if c["backward"] else None
        c["dh"] = _normal(g, T, D, dtype=dt) if c["backward"] and c["pre"] else None
    elif c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        c["x"] = _normal(g, M, K, dtype=torch.bfloat16)
        if c["train"]:
            c["w"] = _normal(g, N, K, std=1.0 / math.sqrt(K), dtype=torch.bfloat16)
            c["dy"] = _normal(g, M, N, std=0.01, dtype=torch.bfloat16)
        else:
            codes, scales = _weights(g, 1, N, K)
            c["w_codes"], c["w_scales"] = codes[0], scales[0]
    else:
        T, E, k, L, F = c["T"], c["E"], c["k"], c["L"], c["F"]
        c["z"] = _normal(g, T, L, dtype=torch.bfloat16)
        # the routing of these tokens, with experts of uneven popularity
        choice = torch.sigmoid(_normal(g, T, E)) + _normal(g, E, std=0.1)
        idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
        perm, counts, offsets, _ = _group(idx, E)
        c["perm"], c["offsets"] = perm, offsets
        c["most"] = max(1, int(counts.max()))
        c["up"], c["down"] = _weights(g, E, F, L), _weights(g, E, L, F)
    return c


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _group(idx, E):
    """(perm, counts, offsets, pos): pairs t*k + j by expert, then by pair."""
    flat = idx.reshape(-1).to(torch.int64)
    perm = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = torch.cumsum(counts, 0)
    pos = torch.empty_like(perm)
    pos[perm] = torch.arange(flat.numel(), device=idx.device)
    return perm.to(torch.int32), counts.to(torch.int32), offsets.to(torch.int32), pos.to(torch.int32)


def _scores(logits, score):
    """Scores in 64 bits (selection compares values that may be next to each
    other), and which logits take part."""
    l = logits.to(torch.float64)
    live = l > -math.inf
    if score == "sigmoid":
        return torch.where(live, 1.0 / (1.0 + torch.exp(-l)), 0.0), live
    top = torch.where(live, l, -math.inf).amax(1, keepdim=True)
    e = torch.where(live, torch.exp(l - torch.where(top > -math.inf, top, 0.0)), 0.0)
    return e / e.sum(1, keepdim=True).clamp_min(1e-300), live


def _route_plain(c):
    logits, T, E, k = c["logits"], c["T"], c["E"], c["k"]
    s64, live = _scores(logits, c["score"])
    s = s64.to(torch.float32)
    choice = s if c["b"] is None else s + c["b"]
    choice = torch.where(live, choice, -math.inf)
    if c["groups"] > 1:
        G = c["groups"]
        two = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values[:, :, :2]
        best = torch.sort(two[:, :, 0] + two[:, :, 1], dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter_(1, best, True)
        choice = torch.where(kept.repeat_interleave(E // G, 1), choice, -math.inf)
    order = torch.sort(choice, dim=1, descending=True, stable=True)
    idx, chosen = order.indices[:, :k], order.values[:, :k] > -math.inf
    p = torch.where(chosen, torch.gather(s, 1, idx), 0.0)
    if c["renorm"]:
        w = p / (p.sum(1, keepdim=True) + RENORM_EPS) * c["scale"]
    else:
        w = p * c["scale"]
    out = [idx.to(torch.int32), w]
    if c["grouping"]:
        out += list(_group(idx, E))
    if c["backward"]:
        p = torch.where(chosen, torch.gather(s64, 1, idx), 0.0)
        u = torch.where(chosen, c["dw"] * c["scale"], 0.0).to(torch.float64)
        if c["renorm"]:
            total = p.sum(1, keepdim=True) + RENORM_EPS
            ds = (u - (u * p).sum(1, keepdim=True) / total) / total
        else:
            ds = u
        full = torch.zeros(T, E, dtype=torch.float64, device=logits.device).scatter_(1, idx, ds)
        if c["score"] == "sigmoid":
            dl = full * s64 * (1.0 - s64)
        else:
            dl = s64 * (full - (full * s64).sum(1, keepdim=True))
        out.append(dl.to(logits.dtype))
    return out


def _rms(v):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + NORM_EPS)


def _norm_plain(c):
    dt = c["x"].dtype
    x, y = c["x"].float(), c["y"].float()
    gate = 1.0 if c["g"] is None else c["g"].float()
    ry = _rms(y) if c["post"] else 1.0
    pw = c["post_w"].float() if c["post"] else 1.0
    n = y * ry * pw
    r = (c["alpha"] * x + gate * n).to(dt)
    out = [r]
    rf = r.float()
    if c["pre"]:
        rr, qw = _rms(rf), c["pre_w"].float()
        out.append((rf * rr * qw).to(dt))
    if not c["backward"]:
        return out
    d = c["dr"].float()
    if c["pre"]:
        dh = c["dh"].float()
        v = dh * qw
        d = d + rr * (v - rf * rr * rr * (v * rf).mean(1, keepdim=True))
    dn = d * gate
    if c["post"]:
        v = dn * pw
        dy = ry * (v - y * ry * ry * (v * y).mean(1, keepdim=True))
    else:
        dy = dn
    out += [(c["alpha"] * d).to(dt), dy.to(dt)]
    if c["post"]:
        out.append((dn * y * ry).sum(0))
    if c["pre"]:
        out.append((dh * rf * rr).sum(0))
    dg = d * n
    if c["gate"] == "channel":
        out.append(dg.sum(0))
    elif c["gate"] == "token":
        out.append(dg.sum(1, keepdim=True))
    elif c["gate"] == "full":
        out.append(dg.to(dt))
    return out


def _pad128(x):
    k = x.shape[-1]
    return torch.nn.functional.pad(x, (0, _blocks(k) * 128 - k))


def _codes(v, amax):
    """v in E4M3, in units of its block's scale, and the scale.  The factor is
    one rounded quotient (a number over a tensor would be two roundings)."""
    amax = amax.clamp_min(F8_FLOOR)
    return (v * (torch.full_like(amax, F8_MAX) / amax)).to(torch.float8_e4m3fn), amax / F8_MAX


def _rows_plain(x):
    """The values that x [M, K] has after a scale for each 128 of a row."""
    M, K = x.shape
    v = _pad128(x.float()).view(M, -1, 128)
    q, s = _codes(v, v.abs().amax(2, keepdim=True))
    return (q.float() * s).view(M, -1)[:, :K]


def _square_plain(w):
    """The values that w [N, K] has after a scale for each 128 x 128 block."""
    N, K = w.shape
    v = torch.nn.functional.pad(_pad128(w.float()), (0, 0, 0, _blocks(N) * 128 - N))
    v = v.view(_blocks(N), 128, _blocks(K), 128)
    q, s = _codes(v, v.abs().amax((1, 3), keepdim=True))
    return (q.float() * s).view(_blocks(N) * 128, -1)[:N, :K]


def _wide(scales, rows, cols):
    return scales.repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]


def _linear_plain(c):
    dt = _dt(c["out"])
    if not c["train"]:
        w = c["w_codes"].float() * _wide(c["w_scales"], c["N"], c["K"])
        return [(_rows_plain(c["x"]) @ w.t()).to(dt)]
    w = _square_plain(c["w"])
    y = (_rows_plain(c["x"]) @ w.t()).to(dt)
    dx = (_rows_plain(c["dy"]) @ w).to(torch.bfloat16)
    dw = _rows_plain(c["dy"].t()) @ _rows_plain(c["x"].t()).t()
    return [y, dx, dw]


def _spaced(c):
    """For each grouped row, its place in a [E, most] grid."""
    off = c["offsets"].to(torch.int64)
    row = torch.arange(c["perm"].numel(), device=off.device)
    e = torch.searchsorted(off, row, right=True) - 1
    return e * c["most"] + row - off[e]


def _experts_plain(c):
    E, L, F, most = c["E"], c["L"], c["F"], c["most"]
    at = _spaced(c)

    def product(rows, mats, n, k):
        codes, scales = mats
        a = torch.zeros(E * most, k, device=rows.device)
        a[at] = rows
        w = codes.float() * _wide(scales, n, k)
        return torch.bmm(a.view(E, most, k), w.transpose(1, 2)).reshape(E * most, n)[at]

    z = _rows_plain(c["z"])[c["perm"].to(torch.int64) // c["k"]]
    h = product(z, c["up"], F, L).to(torch.bfloat16).float()
    h = torch.where(h > 0, h, 0.0)
    return [product(_rows_plain(h * h), c["down"], L, F).to(torch.bfloat16)]


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------
def _route_own(c):
    from latentmoe_expert_routing_b200 import ops
    idx, w = ops.route_topk(c["logits"], c["k"], bias=c["b"], score=c["score"], n_group=c["groups"],
                            topk_group=c["keep"], renorm=c["renorm"], scale=c["scale"])
    out = [idx, w]
    if c["grouping"]:
        counts, offsets, perm, pos = ops.route_group(idx, c["E"])
        out += [perm, counts, offsets, pos]
    if c["backward"]:
        out.append(ops.route_topk_backward(c["logits"], idx, w, c["dw"], score=c["score"],
                                           renorm=c["renorm"], scale=c["scale"]))
    return out


def _norm_own(c):
    from latentmoe_expert_routing_b200 import ops
    f = ops.norm_residual(c["x"], c["y"], post_weight=c["post_w"], gate=c["g"], residual_scale=c["alpha"],
                          pre_weight=c["pre_w"], eps=NORM_EPS, stats=c["backward"])
    out = [f.r] + ([f.h] if c["pre"] else [])
    if c["backward"]:
        b = ops.norm_residual_backward(c["dr"], c["dh"], c["y"], f, post_weight=c["post_w"], gate=c["g"],
                                       residual_scale=c["alpha"], pre_weight=c["pre_w"])
        out += [b.dx, b.dy] + [v for v in (b.dpost_weight, b.dpre_weight, b.dgate) if v is not None]
    return out


def _linear_own(c):
    from latentmoe_expert_routing_b200 import ops
    if not c["train"]:
        w = ops.Fp8(c["w_codes"], c["w_scales"])
        return [ops.gemm_fp8(ops.quantize_fp8(c["x"]), w, out_dtype=c["out"])]
    w, w_t = ops.quantize_fp8_weight(c["w"], transposed=True)
    y = ops.gemm_fp8(ops.quantize_fp8(c["x"]), w, out_dtype=c["out"])
    dx = ops.gemm_fp8(ops.quantize_fp8(c["dy"]), w_t, out_dtype="bf16")
    dw = ops.gemm_fp8(ops.quantize_fp8(c["dy"], transpose=True), ops.quantize_fp8(c["x"], transpose=True),
                      out_dtype="fp32")
    return [y, dx, dw]


def _experts_own(c):
    from latentmoe_expert_routing_b200 import ops
    z = ops.quantize_fp8(c["z"], perm=c["perm"], k=c["k"])
    h = ops.gemm_fp8(z, ops.Fp8(*c["up"]), offsets=c["offsets"], out_dtype="bf16")
    return [ops.gemm_fp8(ops.quantize_fp8(h, relu2=True), ops.Fp8(*c["down"]), offsets=c["offsets"],
                         out_dtype="bf16")]


def run(state):
    if own:
        return {"route": _route_own, "norm": _norm_own, "linear": _linear_own, "experts": _experts_own}[state["op"]](state)
    return {"route": _route_plain, "norm": _norm_plain, "linear": _linear_plain,
            "experts": _experts_plain}[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "route":
        es, P = 2 if c["dtype"] == "bf16" else 4, c["T"] * c["k"]
        b = c["T"] * c["E"] * es + P * 8 + (4 * c["E"] if c["bias"] else 0)
        flops = 6 * c["T"] * c["E"]
        if c["grouping"]:
            b += P * 8 + 8 * c["E"]
        if c["backward"]:
            b += P * 4 + c["T"] * c["E"] * es
            flops += 6 * c["T"] * c["E"]
        return {"bytes": b, "flops": flops}
    if c["op"] == "norm":
        es, n = 2 if c["dtype"] == "bf16" else 4, c["T"] * c["D"]
        full = c["gate"] == "full"
        vecs = (c["post"] + c["pre"] + (c["gate"] == "channel")) * c["D"]
        b = n * es * (3 + c["pre"] + full) + vecs * es
        flops = n * 12
        if c["backward"]:          # the gradients in, x's and y's (and a full gate's) out
            b += n * es * (3 + c["pre"] + full) + vecs * 4
            flops += n * 24
        return {"bytes": b, "flops": flops}
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        es = 2 if c["out"] == "bf16" else 4
        if not c["train"]:
            return {"bytes": M * K * 2 + N * K + _blocks(N) * _blocks(K) * 4 + M * N * es, "flops": 2 * M * N * K}
        return {"bytes": M * K * 4 + N * K * 6 + M * N * (2 + es), "flops": 6 * M * N * K}
    P, E, L, F = c["T"] * c["k"], c["E"], c["L"], c["F"]
    hit = min(E, P)
    return {"bytes": c["T"] * L * 2 + hit * 2 * F * L + P * (4 + 2 * L), "flops": 4 * P * F * L}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _np(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def _exact_route(c):
    T, E, k = c["T"], c["E"], c["k"]
    l, rows = _np(c["logits"]), np.arange(T)[:, None]
    live = np.isfinite(l)
    if c["score"] == "sigmoid":
        s = np.where(live, 1.0 / (1.0 + np.exp(-np.where(live, l, 0.0))), 0.0)
    else:
        top = np.max(np.where(live, l, -np.inf), axis=1, keepdims=True)
        s = np.where(live, np.exp(np.where(live, l - np.where(np.isfinite(top), top, 0.0), 0.0)), 0.0)
        z = s.sum(1, keepdims=True)
        s = np.divide(s, z, out=np.zeros_like(s), where=z > 0)
    # a choice score is a 32-bit number by definition
    choice = s.astype(np.float32)
    if c["b"] is not None:
        choice = choice + c["b"].cpu().numpy()[None]
    choice = np.where(live, choice, np.float32(-np.inf))
    G = c["groups"]
    if G > 1:
        two = np.sort(choice.reshape(T, G, E // G), axis=2)[:, :, -2:]
        best = np.argsort(-(two[:, :, 1] + two[:, :, 0]), axis=1, kind="stable")[:, : c["keep"]]
        kept = np.zeros((T, G), bool)
        kept[rows, best] = True
        choice = np.where(np.repeat(kept, E // G, axis=1), choice, np.float32(-np.inf))
    idx = np.argsort(-choice, axis=1, kind="stable")[:, :k]
    some = np.isfinite(choice[rows, idx])
    p = np.where(some, s[rows, idx], 0.0)
    S = p.sum(1, keepdims=True) + 1e-20 if c["renorm"] else 1.0
    out = [None, p / S * c["scale"]] + ([None] * 4 if c["grouping"] else [])
    if c["backward"]:
        u = np.where(some, _np(c["dw"]) * c["scale"], 0.0)
        if c["renorm"]:
            share = p / S
            ds = (u - (u * share).sum(1, keepdims=True)) / S
        else:
            ds = u
        dl = np.zeros((T, E))
        if c["score"] == "sigmoid":
            dl[rows, idx] = ds * p * (1.0 - p)
        else:
            dl[rows, idx] = ds
            dl = s * (dl - (ds * p).sum(1, keepdims=True))
        out.append(dl)
    return out


def _exact_norm(c):
    """Backward by the chain rule through unit-norm rows u = v / rms(v), whose
    pull-back is (d - u <u, d> / D) / rms(v)."""
    D, f64 = c["D"], torch.float64
    y = c["y"].to(f64)
    gate = torch.ones(1, device=y.device, dtype=f64) if c["g"] is None else c["g"].to(f64)
    rms_y = torch.sqrt(y.pow(2).sum(1, keepdim=True) / D + NORM_EPS) if c["post"] else torch.ones_like(y[:, :1])
    u = y / rms_y
    n = u * c["post_w"].to(f64) if c["post"] else u
    r = c["alpha"] * c["x"].to(f64) + gate * n
    stored = r.to(c["x"].dtype).to(f64)      # the next norm reads the row as it is stored
    rms_r = torch.sqrt(stored.pow(2).sum(1, keepdim=True) / D + NORM_EPS)
    t = stored / rms_r
    out = [r] + ([t * c["pre_w"].to(f64)] if c["pre"] else [])
    if c["backward"]:
        d = c["dr"].to(f64)
        if c["pre"]:
            dh = c["dh"].to(f64)
            dt = dh * c["pre_w"].to(f64)
            d = d + (dt - t * ((dt * t).sum(1, keepdim=True) / D)) / rms_r
        dn = d * gate
        if c["post"]:
            du = dn * c["post_w"].to(f64)
            dy = (du - u * ((du * u).sum(1, keepdim=True) / D)) / rms_y
        else:
            dy = dn
        out += [c["alpha"] * d, dy]
        out += [(dn * u).sum(0)] if c["post"] else []
        out += [(dh * t).sum(0)] if c["pre"] else []
        if c["gate"] != "none":
            dg = d * n
            out.append({"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1, keepdim=True),
                        "full": lambda: dg}[c["gate"]]())
    return out


def _exact_values(x, block_rows):
    """x [R, K] after quantisation in blocks of block_rows x 128, in 64 bits.  A
    block's scale, the factor into its units and the scaled value are 32-bit
    numbers by definition; the rounding to E4M3 is done here on 64-bit numbers:
    three bits behind the leading one, steps of 2^-9 below 2^-6."""
    R, K = x.shape
    pr, pk = -(-R // block_rows) * block_rows, _blocks(K) * 128
    v = torch.zeros(pr, pk, device=x.device, dtype=torch.float32)
    v[:R, :K] = x
    v = v.reshape(pr // block_rows, block_rows, pk // 128, 128)
    top = torch.clamp(v.abs().amax(3, keepdim=True).amax(1, keepdim=True), min=F8_FLOOR)
    t = (v * (torch.tensor(F8_MAX, device=x.device) / top)).to(torch.float64)
    e = torch.clamp(torch.frexp(t).exponent - 1, min=-6).to(torch.float64)
    step = torch.exp2(e - 3.0)
    q = torch.clamp(torch.round(t / step) * step, -F8_MAX, F8_MAX)
    return (q * (top / F8_MAX).to(torch.float64)).reshape(pr, pk)[:R, :K]


def _exact_weights(codes, scales):
    s = scales.to(torch.float64)
    n, k = codes.shape[-2:]
    at = (torch.arange(n, device=s.device) // 128, torch.arange(k, device=s.device) // 128)
    return codes.to(torch.float32).to(torch.float64) * s[..., at[0][:, None], at[1][None, :]]


def _exact_linear(c):
    x = c["x"].float()
    if not c["train"]:
        return [_exact_values(x, 1) @ _exact_weights(c["w_codes"], c["w_scales"]).t()]
    w, dy = _exact_values(c["w"].float(), 128), c["dy"].float()
    return [_exact_values(x, 1) @ w.t(), _exact_values(dy, 1) @ w,
            _exact_values(dy.t(), 1) @ _exact_values(x.t(), 1).t()]


def _exact_experts(c):
    off, tok = c["offsets"].tolist(), c["perm"].long() // c["k"]
    z = _exact_values(c["z"].float(), 1)
    y = torch.zeros(tok.numel(), c["L"], device=z.device, dtype=torch.float64)
    for e in range(c["E"]):
        a, b = off[e], off[e + 1]
        if a < b:
            up = _exact_weights(c["up"][0][e], c["up"][1][e])
            h = (z[tok[a:b]] @ up.t()).to(torch.bfloat16).float().clamp_min(0.0)
            y[a:b] = _exact_values(h * h, 1) @ _exact_weights(c["down"][0][e], c["down"][1][e]).t()
    return [y]


def exact(case, seed):
    c = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "linear": _exact_linear, "experts": _exact_experts}[c["op"]](c)
