"""bf16 results of long contractions of one sign, where a sum that is cut off
after every addition drifts by a part of itself that grows with its length.

The tolerance does not grow with the length.  A result has to be what bf16
makes of some value within 2^-12 of the sum of magnitudes around the exact
one: a quarter of what half a bf16 step (2^-8 of a value, at least 2^-9 of its
upper neighbour) can move a value near a power of two.  What a sum in fp32
chunks needs of it: at most 256 truncating steps in a chunk (256 * 2^-22 = 2^-14)
and one rounding to nearest per chunk, at most 256 chunks of 256 steps
(2^8 * 2^-24 = 2^-16)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SLACK = 2.0 ** -12


def P():
    from second_order_optimizer_shampoo_b200 import prism
    return prism


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def check(got, ref, absum):
    """got (bf16) lies between the roundings of ref - tol and ref + tol; the
    conversion goes through fp32, which moves those bounds by 2^-24 at most."""
    tol = (SLACK + 2.0 ** -23) * absum
    low, high = (ref - tol).to(torch.bfloat16), (ref + tol).to(torch.bfloat16)
    bad = (got.double() < low.double()) | (got.double() > high.double())
    assert int(bad.sum()) == 0, f"{int(bad.sum())} of {bad.numel()}"


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K", [4160, 8192, 65536, 65600, 1 << 20])
def test_grouped_rows(K, trans):
    g = gen(1)
    E, N, edges = 2, 72, [0, 21, 40]
    X = (torch.rand(40, K, generator=g, device="cuda") + 0.5).bfloat16()
    W = (torch.rand(*((E, N, K) if trans else (E, K, N)), generator=g, device="cuda") + 0.5).bfloat16()
    Y = P().shp_grouped_matmul(X, torch.tensor(edges, device="cuda"), W, w_trans=trans)
    for e in range(E):
        w = W[e].double().t() if trans else W[e].double()
        ref = X[edges[e]:edges[e + 1]].double() @ w
        check(Y[edges[e]:edges[e + 1]], ref, ref)


@pytest.mark.parametrize("tall", [64, 128, 256])
def test_grouped_rows_of_each_tile_height(tall):
    """Groups of equal size that fill tiles of 64, 128 and 256 rows."""
    g = gen(2)
    K, N, E = 1 << 18, 264, 2
    T = E * tall
    X = (torch.rand(T, K, generator=g, device="cuda") + 0.5).bfloat16()
    W = (torch.rand(E, K, N, generator=g, device="cuda") + 0.5).bfloat16()
    Y = P().shp_grouped_matmul(X, torch.arange(E + 1, device="cuda") * tall, W)
    ref = torch.bmm(X.view(E, tall, K).double(), W.double()).view(T, N)
    check(Y, ref, ref)


@pytest.mark.parametrize("batch,M,N,K", [(1, 21, 72, 1 << 22), (1, 21, 72, 262144), (1, 21, 72, 16416), (1, 300, 264, 262208),
                                         (40, 21, 72, 1 << 18), (38, 1, 264, 262144 + 96)])
def test_mx4_product(batch, M, N, K):
    """The blocks' scales are spread over 2^-12 to 1, so that the smallest units
    of the products lie far below those of their sum."""
    p = P()
    g = gen(3)

    def operand(rows):
        x = torch.rand(batch, rows, K, generator=g, device="cuda") + 0.5
        e = torch.randint(-12, 1, (batch, rows, K // 32, 1), generator=g, device="cuda")
        return p.shp_mx4_quantize(torch.ldexp(x.unflatten(-1, (-1, 32)), e).flatten(-2).bfloat16())

    A, As = operand(M)
    B, Bs = operand(N)
    C = p.shp_mx4_matmul(A, As, B, Bs)
    for i in range(batch):
        a = p.shp_mx4_dequantize(A[i:i + 1], As[i:i + 1], K)[0].double()
        b = p.shp_mx4_dequantize(B[i:i + 1], Bs[i:i + 1], K)[0].double()
        ref = a @ b.t()
        check(C[i], ref, ref)
