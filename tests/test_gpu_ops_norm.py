"""norm_residual and its gradient on the GPU against 64-bit forms.

fp32 arithmetic: a sum of D squares by per-thread sums of 8 or 16 terms and two
trees of 5 steps is off by at most 30 units of 2^-24, so a reciprocal norm by
16 + 3; a result is a handful of products of these: 32 units of the terms it adds
up.  A bf16 result adds half a step, 2^-8 of its value.  h and the gradients
are compared for the r that the call itself stored, which is what they read.
Sums over T rows: T/blocks terms in a row, then two trees: 32 + T units of the
sum of magnitudes, more than any order needs."""
import pytest
import torch

from tests import ops_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latentmoe_expert_routing_b200 import build
    build.build()
    from latentmoe_expert_routing_b200 import ops
    return ops


def _half(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def _inputs(T, D, dtype, gate, post, pre, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    d = dict(x=n(T, D) * 2, y=n(T, D) * 0.7, dr=n(T, D), dh=n(T, D) if pre else None,
             post=1 + 0.1 * n(D) if post else None, pre=1 + 0.1 * n(D) if pre else None,
             gate={"none": None, "channel": 0.5 + 0.2 * n(D), "token": 0.5 + 0.2 * n(T, 1),
                   "full": 0.5 + 0.2 * n(T, D)}[gate])
    return {k: None if v is None else v.to(dtype).cuda() for k, v in d.items()}


def _within(got, ref, tol, what):
    err = (got.detach().cpu().double() - ref).abs()
    assert got.shape == ref.shape and bool((err <= tol).all()), (what, float((err - tol).max()), float(err.max()))


def _forward(ops, v, alpha, stats=True):
    return ops.norm_residual(v["x"], v["y"], post_weight=v["post"], gate=v["gate"], residual_scale=alpha,
                             pre_weight=v["pre"], eps=EPS, stats=stats)


def _backward(ops, v, alpha, f, dr="dr"):
    return ops.norm_residual_backward(v[dr] if dr else None, v["dh"], v["y"], f, post_weight=v["post"],
                                      gate=v["gate"], residual_scale=alpha, pre_weight=v["pre"])


def _check_forward(v, alpha, f, dtype):
    r = R.norm_r(v["x"], v["y"], v["post"], v["gate"], alpha, EPS)
    big = (alpha * v["x"].cpu().double()).abs() + (r - alpha * v["x"].cpu().double()).abs()
    _within(f.r, r, 32 * U * big + _half(dtype) * r.abs(), "r")
    if v["pre"] is not None:
        h = R.norm_h(f.r, v["pre"], EPS)
        _within(f.h, h, 32 * U * h.abs() + _half(dtype) * h.abs(), "h")


def _formula(v, alpha, r, dr):
    """The gradients in 64 bits for the stored r, and what each is made of."""
    c = lambda t: None if t is None else t.cpu().double()
    y, g = c(v["y"]), c(v["gate"])
    d = c(dr) if dr is not None else torch.zeros_like(y)
    mag = d.abs()
    out, mags = {}, {}
    if v["pre"] is not None:
        r, dh = c(r), c(v["dh"])
        rr, vv = R.rms(r, EPS), dh * c(v["pre"])
        m = (vv * r).mean(1, keepdim=True)
        d = d + rr * (vv - r * rr * rr * m)
        mag = mag + rr * (vv.abs() + r.abs() * rr * rr * (vv * r).abs().mean(1, keepdim=True))
        out["dpre"], mags["dpre"] = (dh * r * rr).sum(0), (dh * r * rr).abs().sum(0)
    gg = 1.0 if g is None else g
    ga = 1.0 if g is None else g.abs()
    if v["post"] is None:
        ry, n, dy, dym = 1.0, y, d * gg, mag * ga
    else:
        w, ry = c(v["post"]), R.rms(y, EPS)
        n, q, qm = y * ry * w, d * gg * w, mag * ga * w.abs()
        dy = ry * (q - y * ry * ry * (q * y).mean(1, keepdim=True))
        dym = ry * (qm + y.abs() * ry * ry * (qm * y.abs()).mean(1, keepdim=True))
        out["dpost"], mags["dpost"] = (d * gg * y * ry).sum(0), (mag * ga * (y * ry).abs()).sum(0)
    out |= {"dx": alpha * d, "dy": dy}
    mags |= {"dx": abs(alpha) * mag, "dy": dym}
    if g is not None:
        dg, dm = d * n, mag * n.abs()
        if g.dim() == 1:
            dg, dm = dg.sum(0), dm.sum(0)
        elif g.shape[1] == 1 and dg.shape[1] > 1:
            dg, dm = dg.sum(1, keepdim=True), dm.sum(1, keepdim=True)
        out["dgate"], mags["dgate"] = dg, dm
    return out, mags


def _check_backward(v, alpha, f, b, dtype, T, dr):
    ref, mag = _formula(v, alpha, f.r, dr)
    got = {"dx": b.dx, "dy": b.dy, "dpost": b.dpost_weight, "dpre": b.dpre_weight, "dgate": b.dgate}
    for n, t in got.items():
        assert (t is None) == (n not in ref), n
        if t is not None:
            half = _half(t.dtype)
            units = 64 if n in ("dx", "dy") or n == "dgate" and t.dim() == 2 else 64 + T
            _within(t, ref[n], units * U * mag[n] + half * ref[n].abs(), n)


SHAPES = [(1, 8), (1, 8192), (3, 64), (64, 8192), (37, 2056), (5, 16384), (300, 256), (700, 1032), (2, 8200)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,D", SHAPES)
def test_both_norms(ops, T, D, gate, dtype):
    v = _inputs(T, D, dtype, gate, True, True, seed=T + D)
    f = _forward(ops, v, 0.5)
    _check_forward(v, 0.5, f, dtype)
    _check_backward(v, 0.5, f, _backward(ops, v, 0.5, f), dtype, T, v["dr"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (False, False)])
def test_one_norm_or_none(ops, gate, post, pre, dtype):
    v = _inputs(50, 520, dtype, gate, post, pre, seed=7)
    f = _forward(ops, v, 1.0)
    assert (f.h is None) == (not pre) and (f.rstd_y is None) == (not post)
    _check_forward(v, 1.0, f, dtype)
    _check_backward(v, 1.0, f, _backward(ops, v, 1.0, f), dtype, 50, v["dr"])


def test_no_gradient_of_r(ops):
    v = _inputs(20, 264, torch.float32, "channel", True, True)
    f = _forward(ops, v, 1.0)
    _check_backward(v, 1.0, f, _backward(ops, v, 1.0, f, dr=None), torch.float32, 20, None)


def test_rows_of_zeros_and_an_infinity(ops):
    v = _inputs(6, 512, torch.float32, "none", True, True)
    v["x"][1], v["y"][1] = 0, 0
    v["x"][2], v["y"][3] = 0, 0
    v["y"][4, 7] = float("inf")
    f = _forward(ops, v, 1.0)
    assert not f.r[1].any() and not f.h[1].any()
    assert torch.equal(f.r[3], v["x"][3])
    assert f.r[4].isnan().any() and f.r[[0, 1, 2, 3, 5]].isfinite().all() and f.h[5].isfinite().all()
    b = _backward(ops, v, 1.0, f)
    assert b.dx[[0, 1, 2, 3, 5]].isfinite().all() and b.dy[[0, 1, 2, 3, 5]].isfinite().all()


@pytest.mark.parametrize("scale", [1e14, 1e-9])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_large_and_small_rows(ops, dtype, scale):
    """|y| = 1e14: ry^3 is below fp32's smallest normal number, the gradient is not."""
    v = _inputs(5, 520, dtype, "channel", True, True, seed=8)
    v["x"], v["y"] = v["x"] * scale, v["y"] * scale
    f = _forward(ops, v, 0.5)
    _check_forward(v, 0.5, f, dtype)
    _check_backward(v, 0.5, f, _backward(ops, v, 0.5, f), dtype, 5, v["dr"])


def test_zero_rows_and_a_tiny_eps(ops):
    """ry = 1e15 for a row of zeros, whose cube no fp32 holds: dy = d g w ry."""
    v = _inputs(3, 264, torch.float32, "token", True, False, seed=9)
    v["y"].zero_()
    f = ops.norm_residual(v["x"], v["y"], post_weight=v["post"], gate=v["gate"], eps=1e-30, stats=True)
    b = ops.norm_residual_backward(v["dr"], None, v["y"], f, post_weight=v["post"], gate=v["gate"])
    assert torch.equal(f.r, v["x"])
    c = lambda t: t.cpu().double()
    ref = c(v["dr"]) * c(v["gate"]) * c(v["post"]) * 1e15
    _within(b.dy, ref, 32 * U * ref.abs(), "dy")
    assert not b.dgate.any() and not b.dpost_weight.any()


def test_against_differences(ops):
    """Directional central differences of the 64-bit function, r kept in fp32:
    its rounding moves h by units of 2^-24 only, which the kernel's own error
    bound covers; truncation h^2 with a third derivative of order one."""
    T, D, step = 4, 64, 1e-4
    v = _inputs(T, D, torch.float32, "channel", True, True, seed=9)
    f = _forward(ops, v, 0.8)
    b = _backward(ops, v, 0.8, f)
    c = {k: t.cpu().double() for k, t in v.items()}

    def loss(x, y, post, gate, pre):
        r = R.norm_r(x, y, post, gate, 0.8, EPS)
        return float((r * c["dr"]).sum() + (R.norm_h(r, pre, EPS) * c["dh"]).sum())

    names = ("x", "y", "post", "gate", "pre")
    grads = dict(x=b.dx, y=b.dy, post=b.dpost_weight, gate=b.dgate, pre=b.dpre_weight)
    for n in names:
        way = torch.randn(c[n].shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
        at = lambda s: loss(*[c[m] + (s * step * way if m == n else 0) for m in names])
        diff = (at(1) - at(-1)) / (2 * step)
        got = float((grads[n].cpu().double() * way).sum())
        scale = float((grads[n].cpu().double() * way).abs().sum())
        assert abs(got - diff) <= 1e-6 * scale + 1e-5, (n, got, diff)


def test_strides_views_and_empty(ops):
    v = _inputs(30, 128, torch.bfloat16, "full", True, True)
    want = _forward(ops, v, 1.0)
    wide = {k: torch.zeros(30, 264, dtype=torch.bfloat16, device="cuda") for k in ("x", "y", "gate")}
    for off in (8, 3):                                          # 3: rows off 16 bytes, copied
        for k in wide:
            wide[k][:, off:off + 128] = v[k]
        w = dict(v, **{k: t[:, off:off + 128] for k, t in wide.items()})
        got = _forward(ops, w, 1.0)
        assert torch.equal(got.r, want.r) and torch.equal(got.h, want.h)
        a, b = _backward(ops, v, 1.0, want), _backward(ops, w, 1.0, got)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    e = _inputs(0, 128, torch.bfloat16, "channel", True, True)
    f = _forward(ops, e, 1.0)
    b = _backward(ops, e, 1.0, f)
    assert f.r.shape == (0, 128) and not b.dpost_weight.any() and not b.dpre_weight.any() and not b.dgate.any()


def test_in_place_through_the_c_call(ops):
    """r over x, h over y; dx over dr, dy over dh."""
    from latentmoe_expert_routing_b200 import binding as B
    v = _inputs(40, 1024, torch.bfloat16, "channel", True, True)
    f = _forward(ops, v, 0.5)
    b = _backward(ops, v, 0.5, f)
    st = torch.cuda.current_stream().cuda_stream
    x, y = v["x"].clone(), v["y"].clone()
    a = B.moe_norm_args(T=40, D=1024, dtype=B.MOE_BF16, gate_kind=B.MOE_GATE_CHANNEL, residual_scale=0.5, eps=EPS,
                        x=x.data_ptr(), ldx=1024, y=y.data_ptr(), ldy=1024, post_weight=v["post"].data_ptr(),
                        pre_weight=v["pre"].data_ptr(), gate=v["gate"].data_ptr(), r=x.data_ptr(), ldr=1024,
                        h=y.data_ptr(), ldh=1024)
    B.moe_norm_residual(a, st)
    assert torch.equal(x, f.r) and torch.equal(y, f.h)
    dr, dh = v["dr"].clone(), v["dh"].clone()
    s = [torch.empty(1024, device="cuda") for _ in range(3)]
    n = B.moe_norm_residual_workspace(40, 1024)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    a = B.moe_norm_args(T=40, D=1024, dtype=B.MOE_BF16, gate_kind=B.MOE_GATE_CHANNEL, residual_scale=0.5, eps=EPS,
                        y=v["y"].data_ptr(), ldy=1024, post_weight=v["post"].data_ptr(),
                        pre_weight=v["pre"].data_ptr(), gate=v["gate"].data_ptr(), r=f.r.data_ptr(), ldr=1024,
                        rstd_y=f.rstd_y.data_ptr(), rstd_r=f.rstd_r.data_ptr(), dr=dr.data_ptr(), lddr=1024,
                        dh=dh.data_ptr(), lddh=1024, dx=dr.data_ptr(), lddx=1024, dy=dh.data_ptr(), lddy=1024,
                        dpost_weight=s[0].data_ptr(), dpre_weight=s[1].data_ptr(), dgate=s[2].data_ptr())
    B.moe_norm_residual_backward(a, ws.data_ptr(), n, st)
    for got, want in zip([dr, dh] + s, b):
        assert torch.equal(got, want)


def test_captured_replayed_and_repeatable(ops):
    v = _inputs(500, 2048, torch.bfloat16, "token", True, True, seed=5)

    def run():
        f = _forward(ops, v, 1.0)
        return tuple(t for t in f if t is not None) + tuple(t for t in _backward(ops, v, 1.0, f) if t is not None)

    first = run()
    assert all(torch.equal(a, b) for a, b in zip(first, run()))          # one order of sums
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                                   # each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    new = _inputs(500, 2048, torch.bfloat16, "token", True, True, seed=6)
    for k, t in v.items():
        t.copy_(new[k])
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for s, (g, _) in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refuses_wrong_tensors(ops):
    v = _inputs(4, 64, torch.float32, "channel", True, True)
    bad = [dict(y=v["y"][:3]), dict(y=v["y"].bfloat16()), dict(post=v["post"][:8]), dict(gate=v["gate"][:8]),
           dict(gate=v["gate"].bfloat16()), dict(pre=v["pre"].cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            _forward(ops, dict(v, **kw), 1.0)
    f = _forward(ops, v, 1.0, stats=False)
    with pytest.raises(ValueError, match="stats"):
        _backward(ops, v, 1.0, f)
    f = _forward(ops, v, 1.0)
    with pytest.raises(ValueError, match="dh"):
        _backward(ops, dict(v, dh=None), 1.0, f)
