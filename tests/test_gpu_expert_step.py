"""One training step of an expert layer through the library: the grouped forward
product, its two gradients, the optimizer's step on the weight blocks, and the
4-bit copy of the updated blocks with the product that reads it.  Every stage
is compared with float64 on what the stage before it produced."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from helpers import U_3XTF32, U_FP32  # noqa: E402


@pytest.mark.parametrize("E,K,N,sizes", [(4, 256, 512, [190, 0, 37, 300]), (2, 72, 264, [1, 64])])
def test_expert_layer_step(E, K, N, sizes):
    from second_order_optimizer_shampoo_b200 import prism as P, synth
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    T = sum(sizes)
    edges = [0]
    for n in sizes:
        edges.append(edges[-1] + n)
    off = torch.tensor(edges, dtype=torch.int64, device="cuda")
    W = rnd(E, K, N) / K ** 0.5  # fp32 master blocks
    Wb = W.to(torch.bfloat16)
    X, dY = rnd(T, K).to(torch.bfloat16), rnd(T, N).to(torch.bfloat16)

    # forward and backward
    Y = P.shp_grouped_matmul(X, off, Wb)
    dX = P.shp_grouped_matmul(dY, off, Wb, w_trans=True, dtype=torch.float32)
    G = P.shp_grouped_wgrad(X, dY, off)
    P.shp_grouped_wgrad(X, dY, off, out=G, accumulate=True)  # a second micro-batch, the same rows
    for e in range(E):
        a, b = edges[e], edges[e + 1]
        x, d, w = X[a:b].double(), dY[a:b].double(), Wb[e].double()
        # tensor-core sums: 2^-22 of the magnitudes per 16 products; stores eps / 2
        tol = K / 16 * 2.0 ** -22 * (x.abs() @ w.abs()) + 2.0 ** -8 * (x @ w).abs()
        assert bool(((Y[a:b].double() - x @ w).abs() <= tol).all())
        tol = 33 * 2.0 ** -22 * (d.abs() @ w.abs().t()) + 2.0 ** -24 * (d @ w.t()).abs()
        assert bool(((dX[a:b].double() - d @ w.t()).abs() <= tol).all())
        ref = 2 * (x.t() @ d)
        tol = 2 * 33 * 2.0 ** -22 * (x.abs().t() @ d.abs()) + 2.0 ** -23 * ref.abs()
        assert bool(((G[e].double() - ref).abs() <= tol).all())

    # the optimizer's step on the blocks, with G as it was written
    L = torch.eye(K, device="cuda").repeat(E, 1, 1) * 1e-2
    R = torch.eye(N, device="cuda").repeat(E, 1, 1) * 1e-2
    L0, R0, W0 = L.double(), R.double(), W.double()
    P.shampoo_gram_ema(G, L, R, 0.9, 1e-3, prec="3xtf32")
    for F, F0, A in ((L, L0, G.double()), (R, R0, G.double().transpose(1, 2))):
        ref = 0.9 * F0 + 0.1 * (A @ A.transpose(1, 2)) + 1e-3 * torch.eye(F.shape[-1], device="cuda").double()
        # beta and 1 - beta are fp32 constants (half an ulp each)
        tol = (2 * U_3XTF32 + (A.shape[2] + 8) * U_FP32) * 0.1 * (A.abs() @ A.abs().transpose(1, 2)) + \
            8 * U_FP32 * (F0.abs() + ref.abs())
        assert bool(((F.double() - ref).abs() <= tol).all())
    roots = []
    for F in (L, R):
        n = F.shape[-1]
        S = torch.from_numpy(synth.sketch_stack(80, n, 8, 7)).cuda()
        root, rep = P.matfn_inv_root(F, "inv4", P.make_opts(d=2, p=8, tol=1e-5, max_iter=40, prec="3xtf32"), S)
        assert bool(torch.isfinite(root).all())
        roots.append(root)
    P.shampoo_apply(W, G, roots[0], roots[1], 1e-3, prec="3xtf32")
    l, r, gg = roots[0].double(), roots[1].double(), G.double()
    ref = W0 - 1e-3 * (l @ gg @ r)
    mag = l.abs() @ gg.abs() @ r.abs()
    assert bool(((W.double() - ref).abs() <= 1e-3 * (4 * U_3XTF32 + (K + N + 8) * U_FP32) * mag + 2 * U_FP32 * (W0.abs() + ref.abs())).all())
    e0 = sizes.index(0) if 0 in sizes else None
    if e0 is not None:  # an expert without rows: no gradient, no step
        assert torch.equal(W[e0].double(), W0[e0])

    # the updated blocks in 4 bits, contracted over K (their rows) as the forward does
    Qt, St = P.shp_mx4_quantize(W, along="rows")
    w4 = P.shp_mx4_dequantize(Qt, St, K).double()  # [E][N][K]
    cap = 48
    A = rnd(E, cap, K).to(torch.bfloat16)
    Qa, Sa = P.shp_mx4_quantize(A)
    a4 = P.shp_mx4_dequantize(Qa, Sa, K, dtype=torch.bfloat16).double()
    C = P.shp_mx4_matmul(Qa, Sa, Qt, St, dtype=torch.float32).double()
    ref = a4 @ w4.transpose(1, 2)
    steps = -(-K // 64)
    tol = (min(steps, 32) * 2.0 ** -22 + 2.0 ** -24) * (a4.abs() @ w4.abs().transpose(1, 2)) + 2.0 ** -24 * ref.abs()
    assert bool(((C - ref).abs() <= tol).all())
    # the 4-bit weights stand for the blocks: at most a quarter of a value's
    # block's largest element off (clipping at 6 of 8; rounding is finer)
    top = W.transpose(1, 2).abs()
    pad = torch.nn.functional.pad(top, (0, -K % 32)).unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)[..., :K]
    assert bool(((w4 - W.transpose(1, 2).double()).abs() <= pad.double() / 4).all())
