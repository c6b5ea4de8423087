"""Operators one behind the other on a stream: a kernel may be launched while the
one before it still runs, and must neither read what that has not written nor
write what it still reads.  Every comparison is bit for bit with the same calls
far apart (a synchronisation between any two)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latentmoe_expert_routing_b200 import build
    build.build()
    from latentmoe_expert_routing_b200 import binding, ops
    return ops, binding


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _quantise(B, x, q):
    M, K = x.shape
    B.moe_quantize_fp8(x.data_ptr(), B.MOE_BF16, M, K, K, None, M, 1, 0, q.codes.data_ptr(), K,
                       q.scales.data_ptr(), M, _stream())


# rows that take the tall form with and without a split of K, and the wide form
@pytest.mark.parametrize("M,N,K", [(8, 1024, 1024), (64, 2048, 4096), (40, 20000, 512), (700, 1024, 768)])
def test_buffers_written_again_at_once(lib, M, N, K):
    """quantise into one buffer, multiply, quantise the next rows into the same
    buffer, multiply, ...: without a wait between them."""
    ops, B = lib
    g = torch.Generator(device="cuda").manual_seed(M)
    xs = [torch.empty(M, K, device="cuda").normal_(generator=g).bfloat16() for _ in range(4)]
    w = ops.quantize_fp8_weight(torch.empty(N, K, device="cuda").normal_(generator=g).bfloat16())
    want = []
    for x in xs:
        q = ops.quantize_fp8(x)
        torch.cuda.synchronize()
        want.append(ops.gemm_fp8(q, w))
        torch.cuda.synchronize()
    q = ops.quantize_fp8(xs[0])
    out = [torch.empty_like(want[0]) for _ in range(40)]
    torch.cuda.synchronize()
    for i, o in enumerate(out):
        _quantise(B, xs[i % 4], q)
        ops.gemm_fp8(q, w, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 4]) for i, o in enumerate(out))


def test_input_overwritten_behind_the_call(lib):
    """the caller's own copies, before and behind a product, on its stream"""
    ops, B = lib
    g = torch.Generator(device="cuda").manual_seed(3)
    xs = [torch.empty(64, 4096, device="cuda").normal_(generator=g).bfloat16() for _ in range(3)]
    w = ops.quantize_fp8_weight(torch.empty(2048, 4096, device="cuda").normal_(generator=g).bfloat16())
    want = []
    for x in xs:
        want.append(ops.gemm_fp8(ops.quantize_fp8(x), w))
        torch.cuda.synchronize()
    x, got = torch.empty_like(xs[0]), []
    for i in range(30):
        x.copy_(xs[i % 3])
        y = ops.gemm_fp8(ops.quantize_fp8(x), w)
        got.append(y.clone())
        y.zero_()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(got))


@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (1000, 64, 6), (16384, 128, 8)])
def test_routes_grouped_at_once(lib, T, E, k):
    ops, B = lib
    g = torch.Generator(device="cuda").manual_seed(T)
    ls = [torch.empty(T, E, device="cuda").normal_(generator=g) for _ in range(3)]
    want = []
    for l in ls:
        idx, w = ops.route_topk(l, k)
        torch.cuda.synchronize()
        want.append((idx, *ops.route_group(idx, E)))
        torch.cuda.synchronize()
    # one buffer for all the results of a kind
    idx, w = torch.empty_like(want[0][0]), torch.empty(T, k, device="cuda")
    counts, offsets, perm, pos = (torch.empty_like(t) for t in want[0][1:])
    ws = torch.empty(max(1, B.moe_route_group_workspace(T, k, E)), dtype=torch.uint8, device="cuda")
    got = []
    for i in range(30):
        B.moe_route_topk(ls[i % 3].data_ptr(), B.MOE_FP32, E, None, T, E, k, B.SCORE["sigmoid"], 1, 1, 1, 1.0,
                         idx.data_ptr(), w.data_ptr(), _stream())
        B.moe_route_group(idx.data_ptr(), T, k, E, counts.data_ptr(), offsets.data_ptr(),
                          perm.data_ptr(), pos.data_ptr(), ws.data_ptr(), ws.numel(), _stream())
        got.append([t.clone() for t in (idx, counts, offsets, perm, pos)])
    torch.cuda.synchronize()
    for i, ts in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(ts, want[i % 3]))


def test_captured_with_forks_and_copies(lib):
    """Nodes in front of an operator that are not kernels (a copy, a memset), and
    more than one of them: two streams join before a product."""
    ops, B = lib
    g = torch.Generator(device="cuda").manual_seed(5)
    M, N, K = 48, 2048, 4096
    src, dy = (torch.empty(M, n, device="cuda").normal_(generator=g).bfloat16() for n in (K, N))
    weight = torch.empty(N, K, device="cuda").normal_(generator=g).bfloat16()
    x = torch.empty_like(src)
    out = torch.empty(M, N, device="cuda")

    def step():
        main, side = torch.cuda.current_stream(), torch.cuda.Stream()
        x.copy_(src)                                            # a copy, then an operator
        fork = torch.cuda.Event()
        fork.record(main)
        side.wait_event(fork)
        with torch.cuda.stream(side):
            w, wt = ops.quantize_fp8_weight(weight, transposed=True)
            join = torch.cuda.Event()
            join.record(side)
        q = ops.quantize_fp8(x)
        main.wait_event(join)                                   # two nodes before the product
        ops.gemm_fp8(q, w, out=out)
        y = out.clone()
        out.zero_()                                             # a memset, then an operator
        dx = ops.gemm_fp8(ops.quantize_fp8(dy), wt, out_dtype="fp32")
        dw = ops.gemm_fp8(ops.quantize_fp8(dy, transpose=True), ops.quantize_fp8(x, transpose=True),
                          out_dtype="fp32")
        return y, dx, dw

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for _ in range(10):
        for t in got:
            t.zero_()
        x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once(lib):
    """the tall form (K split over clusters), the wide form and grouped products of
    two streams beside each other"""
    ops, B = lib
    g = torch.Generator(device="cuda").manual_seed(6)
    n = lambda *s: torch.empty(*s, device="cuda").normal_(generator=g).bfloat16()
    offsets = torch.tensor([0, 100, 100, 420, 600], dtype=torch.int32, device="cuda")
    jobs = [(n(64, 4096), ops.quantize_fp8_weight(n(2048, 4096)), None),
            (n(1500, 1024), ops.quantize_fp8_weight(n(2048, 1024)), None),
            (n(600, 768), ops.quantize_fp8_weight(n(4, 1024, 768)), offsets),
            (n(16, 2048), ops.quantize_fp8_weight(n(10240, 2048)), None)]
    want = [ops.gemm_fp8(ops.quantize_fp8(x), w, offsets=o) for x, w, o in jobs]
    outs = [[torch.empty_like(t) for t in want] for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(40):
        for s, out in zip(streams, outs):
            with torch.cuda.stream(s):
                j = (i + (s is streams[1])) % 4
                x, w, o = jobs[j]
                ops.gemm_fp8(ops.quantize_fp8(x), w, offsets=o, out=out[j])
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    B.moe_sync(None, _stream())
