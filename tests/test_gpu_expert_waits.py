"""The bounded waits of the grouped and 4-bit kernels: one wait of a real launch
runs out (about 10 ms), the kernel records SHP_ETIMEOUT and unwinds with its
copies landed and tensor memory freed, and ordinary calls right after it are
correct."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ETIMEOUT = 19


@pytest.mark.parametrize("which", ["grouped", "wgrad", "mx4_quantize", "mx4_matmul"])
def test_wait_runs_out_and_the_context_survives(which):
    from second_order_optimizer_shampoo_b200 import prism as P
    for _ in range(2):
        status, _ = P.selftest_bounded_wait(which)
        assert status == ETIMEOUT
    torch.cuda.synchronize()  # raises on a sticky error
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    X = torch.randn(5000, 256, generator=g, device="cuda").bfloat16()
    W = torch.randn(20, 256, 512, generator=g, device="cuda").bfloat16()
    off = torch.arange(21, device="cuda") * 250
    Y = P.shp_grouped_matmul(X, off, W, dtype=torch.float32)
    ref = torch.bmm(X.view(20, 250, 256).double(), W.double()).view(5000, 512)
    assert float((Y.double() - ref).norm() / ref.norm()) <= 1e-6
    G = P.shp_grouped_wgrad(X, X, off)
    ref = torch.bmm(X.view(20, 250, 256).double().transpose(1, 2), X.view(20, 250, 256).double())
    assert float((G.double() - ref).norm() / ref.norm()) <= 1e-6
    Q, S = P.shp_mx4_quantize(X)
    v = P.shp_mx4_dequantize(Q, S, 256).double()
    C = P.shp_mx4_matmul(Q, S, Q[:, :1000].contiguous(), S[:, :8].contiguous(), dtype=torch.float32)
    ref = v @ v[:, :1000].transpose(1, 2)
    assert float((C.double() - ref).norm() / ref.norm()) <= 1e-6
