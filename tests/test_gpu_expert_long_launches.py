"""Launches of the grouped and 4-bit products that last many times the limit of
a wait: waits that span a tile or the launch follow the work, so none runs out
and the result is complete."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["grouped_long", "wgrad_long", "mx4_matmul_long"])
def test_no_wait_runs_out_in_a_long_launch(which):
    """Waits of 50 us at most, launches of 1.0, 1.4 and 0.13 ms, steps below 20 us."""
    from second_order_optimizer_shampoo_b200 import prism as P
    for _ in range(3):
        status, _ = P.selftest_bounded_wait(which)
        assert status == 0


def test_long_tiles_of_many_stages_are_complete():
    """Tiles of 8192 stages, several per SM pair, against the sums of ones."""
    from second_order_optimizer_shampoo_b200 import prism as P
    T, m = 1 << 19, 8
    X = torch.ones(T, m, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, T] * 100, device="cuda")  # a decreasing pair counts as an empty group
    G = P.shp_grouped_wgrad(X, X, off)
    assert bool((G[0::2] == T).all()) and not bool(G[1::2].any())
