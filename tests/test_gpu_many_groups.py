"""The most groups the grouped products take, nearly all of them empty or of a
row or two."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 1000, 70000])
def test_65535_groups(T):
    from second_order_optimizer_shampoo_b200 import prism as P
    E, K, N = 65535, 64, 72
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    of = torch.randint(0, E, (T,), generator=g, device="cuda").sort().values  # a row's group
    of[-1] = E - 1
    off = torch.searchsorted(of, torch.arange(E + 1, device="cuda")).contiguous()
    X = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    B = torch.randn(T, N, generator=g, device="cuda").bfloat16()
    W = torch.randn(E, K, N, generator=g, device="cuda").bfloat16()
    Y = P.shp_grouped_matmul(X, off, W, dtype=torch.float32)
    # 64 products in four tensor-core steps of at most 2^-22 of the magnitudes each
    for at in torch.arange(T, device="cuda").split(8192):
        x, w = X[at].double(), W[of[at]].double()
        ref = torch.bmm(x[:, None], w)[:, 0]
        tol = 5 * 2.0 ** -22 * torch.bmm(x.abs()[:, None], w.abs())[:, 0]
        assert bool(((Y[at].double() - ref).abs() <= tol).all())
    G = P.shp_grouped_wgrad(X, B, off)
    ref = torch.zeros_like(G)
    for at in torch.arange(T, device="cuda").split(8192):
        ref.index_add_(0, of[at], X[at].float()[:, :, None] * B[at].float()[:, None, :])
    # at most a few rows per group: each product and sum off by 2^-22 of the magnitudes
    mag = torch.zeros_like(G)
    for at in torch.arange(T, device="cuda").split(8192):
        mag.index_add_(0, of[at], X[at].float().abs()[:, :, None] * B[at].float().abs()[:, None, :])
    assert bool(((G - ref).abs() <= 3 * 2.0 ** -22 * mag).all())
