"""Parity of the expert-grouped products with float64.

Error bounds.  Products of bf16 values are exact in fp32; a tensor-core step
adds 16 of them to the accumulator with truncation, at most 2^-22 of the sum
of magnitudes so far (one ulp for the sum, one for the alignment of the
addends).  bf16 results take the whole contraction in one accumulator, K / 16
steps; fp32 results at most 32 steps, then one rounding (2^-24) per chunk of
512.  The store rounds to the result's type: eps / 2 of the value."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U_STEP = 2.0 ** -22


def P():
    from second_order_optimizer_shampoo_b200 import prism
    return prism


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def offs(edges):
    return torch.tensor(edges, dtype=torch.int64, device="cuda")


def bound(absum, ref, K, dtype):
    steps = -(-K // 16)
    if dtype == torch.float32:
        return (min(steps, 32) * U_STEP + (-(-K // 512)) * 2.0 ** -24) * absum + 2.0 ** -24 * ref.abs()
    return steps * U_STEP * absum + torch.finfo(dtype).eps / 2 * ref.abs()


def check_rows(X, edges, W, trans, Y, Y0):
    """Every row of every group against float64; rows of no group unchanged."""
    covered = torch.zeros(X.shape[0], dtype=torch.bool, device="cuda")
    for e in range(W.shape[0]):
        a, b = edges[e], edges[e + 1]
        if a >= b:
            continue
        covered[a:b] = True
        w = W[e].double().t() if trans else W[e].double()
        ref = X[a:b].double() @ w
        tol = bound(X[a:b].double().abs() @ w.abs(), ref, X.shape[1], Y.dtype)
        assert bool(((Y[a:b].double() - ref).abs() <= tol).all()), f"group {e}"
    assert torch.equal(Y[~covered], Y0[~covered])


SPLITS = {
    "one row": (1, [0, 1]),
    "one group": (700, [0, 700]),
    "empty ends": (300, [0, 0, 0, 130, 130, 300, 300]),
    "ones": (9, [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]),
    "all empty": (5, [0, 0, 0]),
    "padded": (600, [17, 200, 456, 571]),
    "edges": (1281, [0, 255, 511, 768, 1024, 1281]),
    "many": (400, sorted([(i * 397) % 401 for i in range(70)])),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("split", list(SPLITS))
def test_rows_splits(split, trans, dtype):
    T, edges = SPLITS[split]
    K, N = 200, 328
    g = gen(1)
    E = len(edges) - 1
    X, W = rnd(g, T, K), rnd(g, E, *((N, K) if trans else (K, N)), scale=0.1)
    Y = torch.randn(T, N, generator=g, device="cuda").to(dtype)
    Y0 = Y.clone()
    out = P().shp_grouped_matmul(X, offs(edges), W, w_trans=trans, out=Y)
    assert out is Y
    check_rows(X, edges, W, trans, Y, Y0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,K,N", [(600, 8, 8), (600, 1032, 8), (600, 8, 520), (513, 576, 264), (2000, 2048, 1024),
                                   (40, 64, 2056), (1500, 4104, 512)])
def test_rows_sizes(T, K, N, trans, dtype):
    g = gen(2)
    edges = [0, T // 7, T // 7, T // 2, T]
    X, W = rnd(g, T, K), rnd(g, 4, *((N, K) if trans else (K, N)), scale=0.1)
    Y = P().shp_grouped_matmul(X, offs(edges), W, w_trans=trans, dtype=dtype)
    check_rows(X, edges, W, trans, Y, Y)


def check_wgrad(A, B, edges, G, G0=None):
    for e in range(G.shape[0]):
        a, b = edges[e], max(edges[e], edges[e + 1])
        x, y = A[a:b].double(), B[a:b].double()
        ref = x.t() @ y
        tol = bound(x.abs().t() @ y.abs(), ref, max(1, b - a), torch.float32)
        if G0 is not None:
            ref = ref + G0[e].double()
            tol = tol + 2.0 ** -24 * (ref.abs() + G0[e].double().abs())
        assert bool(((G[e].double() - ref).abs() <= tol).all()), f"group {e}"
        if a == b:
            assert torch.equal(G[e], G0[e] if G0 is not None else torch.zeros_like(G[e]))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("split", list(SPLITS))
def test_wgrad_splits(split, accumulate):
    T, edges = SPLITS[split]
    g = gen(3)
    A, B = rnd(g, T, 200), rnd(g, T, 328)
    G0 = torch.randn(len(edges) - 1, 200, 328, generator=g, device="cuda")
    G = P().shp_grouped_wgrad(A, B, offs(edges), out=G0.clone(), accumulate=accumulate)
    check_wgrad(A, B, edges, G, G0 if accumulate else None)


@pytest.mark.parametrize("T,m,n", [(65, 8, 8), (1000, 264, 8), (1000, 8, 520), (3001, 1024, 256), (20000, 128, 136)])
def test_wgrad_sizes(T, m, n):
    g = gen(4)
    edges = [0, 1, T // 3, T // 3, T]
    A, B = rnd(g, T, m), rnd(g, T, n)
    check_wgrad(A, B, edges, P().shp_grouped_wgrad(A, B, offs(edges)))


def test_wgrad_no_rows():
    A = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    G = P().shp_grouped_wgrad(A, A, offs([0, 0, 0]), out=torch.ones(2, 64, 64, device="cuda"))
    assert torch.equal(G, torch.zeros_like(G))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_neighbours_non_finite_rows_stay_out(bad):
    """A group's rows that hold NaN or Inf reach that group's results alone."""
    g = gen(5)
    T, edges = 300, [0, 70, 171, 300]
    A, B, W = rnd(g, T, 136), rnd(g, T, 200), rnd(g, 3, 136, 200)
    A[70:171] = bad
    B[70:171] = bad
    G = P().shp_grouped_wgrad(A, B, offs(edges))
    for e in (0, 2):
        check_wgrad(A[edges[e]:edges[e + 1]], B[edges[e]:edges[e + 1]], [0, edges[e + 1] - edges[e]], G[e:e + 1])
    assert not bool(G[1].isfinite().any())
    Y = P().shp_grouped_matmul(A, offs(edges), W, dtype=torch.float32)
    assert bool(Y[:70].isfinite().all()) and bool(Y[171:].isfinite().all())
    assert not bool(Y[70:171].isfinite().any())


@pytest.mark.parametrize("edges", [[-50, 30, 90, 4000], [0, 80, 40, 100], [200, 300, 1 << 40, -(1 << 40)]])
def test_offsets_out_of_range_are_clamped(edges):
    g = gen(6)
    T = 100
    X, W = rnd(g, T, 64), rnd(g, 3, 64, 72)
    pad = torch.full((3 * T, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = pad[T:2 * T]
    P().shp_grouped_matmul(X, offs(edges), W, out=Y)
    assert bool((pad[:T] == 7).all()) and bool((pad[2 * T:] == 7).all())
    clamp = [min(max(e, 0), T) for e in edges]
    G = P().shp_grouped_wgrad(X, X, offs(edges))
    check_wgrad(X, X, clamp, G)


def test_far_rows():
    """Element offsets beyond 2^31: the groups sit at the end of 4.8 GB of rows."""
    K, N, T = 8192, 8192, 290000
    g = gen(7)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    Y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    a = T - 301
    X[a:] = rnd(g, T - a, K)
    edges = [a, a + 100, T]
    W = rnd(g, 2, K, N, scale=0.02)
    P().shp_grouped_matmul(X, offs(edges), W, out=Y)
    assert not bool(Y[:a].any())
    check_rows(X[a:], [0, 100, 301], W, False, Y[a:], Y[a:])
    del W
    G = P().shp_grouped_wgrad(X, Y, offs(edges))
    check_wgrad(X[a:], Y[a:], [0, 100, 301], G)


def test_repeats_are_identical_and_streams_independent():
    g = gen(8)
    T, K, N, E = 3000, 520, 776, 9
    edges = [0] + sorted(torch.randint(0, T, (E - 1,), generator=torch.Generator().manual_seed(3)).tolist()) + [T]
    X, W, B = rnd(g, T, K), rnd(g, E, K, N, scale=0.1), rnd(g, T, N)
    off = offs(edges)
    Y1, G1 = P().shp_grouped_matmul(X, off, W), P().shp_grouped_wgrad(X, B, off)
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:  # both calls at once on two streams
        with torch.cuda.stream(s):
            for _ in range(3):
                outs.append((P().shp_grouped_matmul(X, off, W), P().shp_grouped_wgrad(X, B, off)))
    torch.cuda.synchronize()
    for y, gr in outs:
        assert torch.equal(y, Y1) and torch.equal(gr, G1)


@pytest.mark.parametrize("T,E,K,N", [(20000, 200, 136, 520), (15000, 300, 72, 328), (70000, 16, 64, 1032)])
def test_more_tiles_than_sm_pairs(T, E, K, N):
    """Tiles handed out at run time, the groups sorted by size (up to 256 of
    them) or not, some empty, sizes far apart; and every repeat the same."""
    g = gen(12)
    p = torch.rand(E, generator=torch.Generator().manual_seed(4)).pow(6)
    sizes = torch.bincount(torch.multinomial(p, T, replacement=True, generator=torch.Generator().manual_seed(5)),
                           minlength=E).tolist()
    edges = [0]
    for n in sizes:
        edges.append(edges[-1] + n)
    assert 0 in sizes and max(sizes) > 256
    X, W, B = rnd(g, T, K), rnd(g, E, K, N, scale=0.1), rnd(g, T, N)
    off = offs(edges)
    for dtype in (torch.bfloat16, torch.float32):
        Y = P().shp_grouped_matmul(X, off, W, dtype=dtype)
        check_rows(X, edges, W, False, Y, Y)
        for _ in range(3):
            assert torch.equal(P().shp_grouped_matmul(X, off, W, dtype=dtype), Y)
    G = P().shp_grouped_wgrad(X, B, off)
    check_wgrad(X, B, edges, G)
    for _ in range(3):
        assert torch.equal(P().shp_grouped_wgrad(X, B, off), G)


def test_two_captured_graphs_at_once():
    """Two graphs of the same calls on other tensors, replayed together on two
    streams: nothing is shared between them."""
    g = gen(13)
    T, K, N, E = 6000, 264, 520, 40
    edges = [0] + sorted(torch.randint(0, T, (E - 1,), generator=torch.Generator().manual_seed(6)).tolist()) + [T]
    off = offs(edges)
    sides = []
    for _ in range(2):
        X, W, B = rnd(g, T, K), rnd(g, E, K, N, scale=0.1), rnd(g, T, N)
        Y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
        G = torch.zeros(E, K, N, device="cuda")
        graph = torch.cuda.CUDAGraph()
        P().shp_grouped_matmul(X, off, W, out=Y)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            P().shp_grouped_matmul(X, off, W, out=Y)
            P().shp_grouped_wgrad(X, B, off, out=G)
        sides.append((graph, X, W, B, Y, G))
    streams = [torch.cuda.Stream() for _ in sides]
    for _ in range(5):
        for s, side in zip(streams, sides):
            with torch.cuda.stream(s):
                side[0].replay()
    torch.cuda.synchronize()
    for _, X, W, B, Y, G in sides:
        check_rows(X, edges, W, False, Y, Y)
        check_wgrad(X, B, edges, G)


def test_captured_calls_follow_the_offsets():
    """A captured graph reads the offsets on the device: a replay with other
    boundaries and rows gives their results."""
    g = gen(9)
    T, K, N, E = 900, 264, 328, 4
    X, W, B = rnd(g, T, K), rnd(g, E, K, N, scale=0.1), rnd(g, T, N)
    off = offs([0, 100, 300, 300, 900])
    Y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    G = torch.zeros(E, K, N, device="cuda")

    def step():
        P().shp_grouped_matmul(X, off, W, out=Y)
        P().shp_grouped_wgrad(X, B, off, out=G)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for edges in ([0, 1, 500, 777, 900], [0, 0, 0, 899, 900]):
        off.copy_(offs(edges))
        X.copy_(rnd(g, T, K))
        graph.replay()
        torch.cuda.synchronize()
        check_rows(X, edges, W, False, Y, Y)
        check_wgrad(X, B, edges, G)


def test_gradients_against_differences():
    """dX and G are the gradients of sum(C * Y): a central difference along a
    random direction, in float64 through the forward formula."""
    g = gen(10)
    T, K, N, E = 200, 64, 72, 3
    edges = [0, 50, 50, 200]
    X, W, C = rnd(g, T, K), rnd(g, E, K, N, scale=0.1), rnd(g, T, N)
    off = offs(edges)
    dX = P().shp_grouped_matmul(C, off, W, w_trans=True, dtype=torch.float32).double()
    dW = P().shp_grouped_wgrad(X, C, off).double()

    def loss(x, w):
        return sum((C[a:b].double() * (x[a:b] @ w[e])).sum() for e, (a, b) in enumerate(zip(edges, edges[1:])))

    x, w, h = X.double(), W.double(), 1e-4
    vx, vw = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64), torch.randn(
        w.shape, generator=g, device="cuda", dtype=torch.float64)
    for got, d in (((dX * vx).sum(), (loss(x + h * vx, w) - loss(x - h * vx, w)) / (2 * h)),
                   ((dW * vw).sum(), (loss(x, w + h * vw) - loss(x, w - h * vw)) / (2 * h))):
        # the loss is linear in each argument, so the difference is exact up to
        # float64 rounding; the gradients carry the fp32 sums' errors
        scale = (dX.abs() * vx.abs()).sum() + (dW.abs() * vw.abs()).sum()
        assert abs(float(got - d)) <= 1e-5 * float(scale)


def test_binding_refuses_wrong_tensors():
    g = gen(11)
    X, W, off = rnd(g, 10, 64), rnd(g, 2, 64, 72), offs([0, 4, 10])
    p = P()
    with pytest.raises(ValueError):
        p.shp_grouped_matmul(X.float(), off, W)
    with pytest.raises(ValueError):
        p.shp_grouped_matmul(X, off.int(), W)
    with pytest.raises(ValueError):
        p.shp_grouped_matmul(X, off[:2], W)
    with pytest.raises(ValueError):
        p.shp_grouped_matmul(X, off, W, w_trans=True)
    with pytest.raises(ValueError):
        p.shp_grouped_matmul(X, off, W, dtype=torch.float16)
    with pytest.raises(ValueError):
        p.shp_grouped_matmul(X.t().contiguous().t(), off, W)
    with pytest.raises(ValueError):
        p.shp_grouped_wgrad(X, X[:5], off)
    with pytest.raises(ValueError):
        p.shp_grouped_wgrad(X, X, off, accumulate=True)
    with pytest.raises(RuntimeError):
        p.shp_grouped_matmul(rnd(g, 10, 60), off, rnd(g, 2, 60, 72))
