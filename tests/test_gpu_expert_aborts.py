"""Launches of the grouped and 4-bit kernels that give up right after their
producers started, with ordinary calls queued directly behind them: copies still
in flight would land in the shared memory of those."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ETIMEOUT = 19


@pytest.mark.parametrize("which", ["grouped", "wgrad", "mx4_quantize", "mx4_matmul"])
def test_calls_behind_an_abort_are_correct(which):
    from second_order_optimizer_shampoo_b200 import _abi as A, prism as P
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    X = torch.randn(3000, 264, generator=g, device="cuda").bfloat16()
    W = torch.randn(12, 264, 520, generator=g, device="cuda").bfloat16()
    off = torch.tensor([250 * i for i in range(13)], device="cuda")

    def calls():
        Q, S, Qt, St = P.shp_mx4_quantize(X, along="both")
        return (P.shp_grouped_matmul(X, off, W), P.shp_grouped_wgrad(X, X, off), Q, S, Qt, St,
                P.shp_mx4_matmul(Q, S, Q, S, dtype=torch.float32))

    want = calls()
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    ws = torch.empty(A.SHP_SELFTEST_WS_BYTES, dtype=torch.uint8, device="cuda")
    code = getattr(A, "SHP_SELFTEST_" + which.upper())
    for _ in range(10):
        for _ in range(2):
            assert A.lib().shp_selftest_bounded_wait(code, status.data_ptr(), None, ws.data_ptr(), ws.numel(),
                                                     torch.cuda.current_stream().cuda_stream) == A.SHP_OK
        got = calls()
        assert int(status.item()) == ETIMEOUT
        for a, b in zip(got, want):
            assert torch.equal(a, b)
