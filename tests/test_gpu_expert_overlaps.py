"""The binding's refusal of results that share memory with an operand, and its
acceptance of neighbours in one buffer."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_out_over_an_operand_is_refused_and_beside_it_is_not():
    from second_order_optimizer_shampoo_b200 import prism as P
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    buf = torch.randn(300, 128, generator=g, device="cuda").bfloat16()
    X = buf[100:200]
    W = torch.randn(2, 128, 128, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, 30, 100], device="cuda")
    want = P.shp_grouped_matmul(X, off, W)
    before = buf.clone()
    for out in (X, buf[1:101], buf[199:299], W[0, :100]):
        with pytest.raises(RuntimeError):
            P.shp_grouped_matmul(X, off, W, out=out)
    assert torch.equal(buf, before)
    assert torch.equal(P.shp_grouped_matmul(X, off, W, out=buf[:100]), want)
    assert torch.equal(P.shp_grouped_matmul(X, off, W, out=buf[200:]), want)
    Q, S = P.shp_mx4_quantize(W)  # operands may be the same
    C = P.shp_mx4_matmul(Q, S, Q, S, dtype=torch.float32)
    assert torch.equal(C, C.transpose(1, 2))
