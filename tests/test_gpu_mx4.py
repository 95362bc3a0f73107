"""MXFP4 quantisation, its inverse and the product, against plain forms.

Quantisation is exact: codes and scale bytes must be equal, ties, saturation,
zero blocks, subnormals and non-finite values included.  The product's bound:
products of codes and scales are exact; a tensor-core step adds 64 of them to
the fp32 accumulator with truncation, at most 2^-22 of the sum of magnitudes
(one ulp for the sum, one for the alignment of the addends); fp32 results take
32 steps per chunk and round (2^-24) once per chunk of 2048; the store rounds
to the type, eps / 2 of the value."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
MID = (GRID[1:] + GRID[:-1]) / 2


def P():
    from second_order_optimizer_shampoo_b200 import prism
    return prism


def ref_quantize(x):
    """Codes [.., cols up to 32] and scale bytes [.., blocks], float64 NumPy."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[-1]
    p = np.zeros(x.shape[:-1] + ((n + 31) // 32 * 32,))
    p[..., :n] = x
    b = p.reshape(p.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    top = np.where(bad, 0, np.abs(np.where(np.isfinite(b), b, 0)).max(-1))
    e = np.frexp(top)[1] - 1 - 2
    sb = np.where(top > 0, np.clip(e + 127, 0, 254), 0)
    y = np.where(bad[..., None], 0, b) / np.exp2(sb - 127.0)[..., None]
    a = np.abs(y)
    code = np.zeros(a.shape, dtype=np.uint8)
    for i, m in enumerate(MID):  # at a midpoint the even code wins
        code += ((a > m) if i % 2 == 0 else (a >= m)).astype(np.uint8)
    code |= (np.signbit(y) & ~bad[..., None]).astype(np.uint8) << 3
    return code.reshape(p.shape), np.where(bad, 255, sb).astype(np.uint8)


def ref_values(code, sb):
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(sb == 255, np.nan, np.exp2(sb.astype(np.float64) - 127))
    return (v.reshape(v.shape[:-1] + (-1, 32)) * s[..., None]).reshape(v.shape)


def unpack(Q):
    q = Q.cpu().numpy()
    out = np.empty(q.shape[:-1] + (q.shape[-1] * 2,), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = q & 15, q >> 4
    return out


def untile(S, rows, blocks):
    """Scale bytes [batch, rows, blocks] by the layout's formula, and whether
    every byte outside them is zero."""
    s = S.cpu().numpy()
    full = np.zeros((s.shape[0], s.shape[1] * 128, s.shape[2] * 4), dtype=np.uint8)
    r, k = np.meshgrid(np.arange(full.shape[1]), np.arange(full.shape[2]), indexing="ij")
    full = s[:, r // 128, k // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4]
    rest = full.copy()
    rest[:, :rows, :blocks] = 0
    return full[:, :rows, :blocks], not rest.any()


def check_quantized(x, Q, S):
    code, sb = ref_quantize(x)
    got, clean = untile(S, x.shape[1], sb.shape[-1])
    assert clean
    np.testing.assert_array_equal(got, sb)
    np.testing.assert_array_equal(unpack(Q), code)


def rand(shape, seed, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(3 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    x *= torch.rand(shape[:-1] + (1,), generator=g, device="cuda") > 0.05  # zero rows
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 8), (1, 1, 4096), (3, 33, 40), (2, 128, 128), (1, 129, 136),
                                             (2, 300, 264), (1, 1000, 520), (5, 7, 1032)])
def test_quantize(batch, rows, cols, dtype):
    X = rand((batch, rows, cols), 1, dtype)
    Q, S, Qt, St = P().shp_mx4_quantize(X, along="both")
    x = X.float().cpu().numpy()
    check_quantized(x, Q, S)
    check_quantized(x.transpose(0, 2, 1), Qt, St)
    for a, (q, s) in (("cols", (Q, S)), ("rows", (Qt, St))):  # one orientation alone
        q1, s1 = P().shp_mx4_quantize(X, along=a)
        assert torch.equal(q1, q) and torch.equal(s1, s)
    for t in (torch.float32, torch.bfloat16):
        V = P().shp_mx4_dequantize(Q, S, cols, dtype=t)
        Vt = P().shp_mx4_dequantize(Qt, St, rows, dtype=t)
        np.testing.assert_array_equal(V.float().cpu().numpy(), ref_values(*ref_quantize(x))[..., :cols])
        np.testing.assert_array_equal(Vt.float().cpu().numpy(),
                                      ref_values(*ref_quantize(x.transpose(0, 2, 1)))[..., :rows])


def test_quantize_special_values():
    """Ties, the clipped interval (6, 8), one step around every midpoint and
    power of two, signed zeros, subnormals, the largest values, NaN and Inf."""
    base = np.float32([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.999, 4])
    near = np.concatenate([np.nextafter(base, np.float32(9)), np.nextafter(base, np.float32(-9))])
    vals = np.concatenate([base, near])
    rows = []
    for scale in (1.0, 2.0 ** -20, 2.0 ** 100, 2.0 ** -120, 2.0 ** -126, 2.0 ** -130):
        for v in vals:
            for peak in (4.0, 7.5):
                r = np.zeros(32, dtype=np.float32)
                r[0], r[1], r[31] = peak * scale, v * scale, -v * scale
                rows.append(r)
    tiny = np.float32(1e-45)
    for v in (tiny, -tiny, 2.0 ** -127, 2.0 ** -128, 2.0 ** -129, 2.0 ** -130, 3e38, -3.4028235e38,
              float("nan"), float("inf"), -float("inf"), -0.0):
        r = np.full(32, -0.0, dtype=np.float32)
        r[5] = v
        rows.append(r)
    x = np.stack(rows)[None]
    X = torch.from_numpy(x).cuda()
    Q, S, Qt, St = P().shp_mx4_quantize(X, along="both")
    check_quantized(x, Q, S)
    check_quantized(x.transpose(0, 2, 1), Qt, St)
    V = P().shp_mx4_dequantize(Q, S, 32).cpu().numpy()
    np.testing.assert_array_equal(V, ref_values(*ref_quantize(x)))  # NaN where the scale is NaN


@pytest.mark.parametrize("cols", [1, 31, 33, 129])
def test_dequantize_any_columns(cols):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    Q = torch.randint(0, 256, (2, 70, (cols + 31) // 32 * 16), generator=g, device="cuda", dtype=torch.uint8)
    S = torch.randint(0, 255, (2, 1, (cols + 127) // 128, 512), generator=g, device="cuda", dtype=torch.uint8)
    sb, _ = untile(S, 70, (cols + 31) // 32)
    ref = ref_values(unpack(Q), sb)[..., :cols]
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(P().shp_mx4_dequantize(Q, S, cols).cpu().numpy(), ref.astype(np.float32))
    V = P().shp_mx4_dequantize(Q, S, cols, dtype=torch.bfloat16)
    np.testing.assert_array_equal(V.float().cpu().numpy(), torch.from_numpy(ref).to(torch.bfloat16).float().numpy())


def operand(batch, rows, K, seed):
    Q, S = P().shp_mx4_quantize(rand((batch, rows, K), seed, torch.float32))
    return Q, S, P().shp_mx4_dequantize(Q, S, Q.shape[2] * 2).double()


def check_product(C, a, b):
    ref = a @ b.transpose(1, 2)
    absum = a.abs() @ b.abs().transpose(1, 2)
    steps = -(-a.shape[2] // 64)
    if C.dtype == torch.float32:
        tol = (min(steps, 32) * 2.0 ** -22 + -(-steps // 32) * 2.0 ** -24) * absum + 2.0 ** -24 * ref.abs()
    else:
        tol = steps * 2.0 ** -22 * absum + torch.finfo(C.dtype).eps / 2 * ref.abs()
    err = (C.double() - ref).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,M,N,K", [(1, 1, 8, 32), (1, 128, 256, 64), (1, 256, 256, 256), (2, 256, 256, 512),
                                         (1, 16, 512, 1024), (3, 300, 1000, 1376), (1, 129, 136, 96),
                                         (2, 513, 264, 2080), (1, 1000, 520, 4192), (1, 4096, 2048, 1024), (40, 64, 72, 160)])
def test_product(batch, M, N, K, dtype):
    A, As, a = operand(batch, M, K, 3)
    B, Bs, b = operand(batch, N, K, 4)
    C = P().shp_mx4_matmul(A, As, B, Bs, dtype=dtype)
    check_product(C, a, b)
    assert torch.equal(P().shp_mx4_matmul(A, As, B, Bs, dtype=dtype), C)


def test_product_picks_every_scale():
    """One nonzero block of A at a time against ones: the scale of every row
    and block, in its own place (powers of two, so the result is exact)."""
    M, N, K = 384, 264, 544
    rows, blocks = np.arange(M)[:, None], np.arange(K // 32)[None, :]
    exps = ((rows * 7 + blocks * 5) % 23 - 11).astype(np.float64)
    for k in range(K // 32):
        a = np.zeros((1, M, K), dtype=np.float32)
        a[0, :, k * 32] = np.exp2(exps[:, k])
        A, As = P().shp_mx4_quantize(torch.from_numpy(a).cuda())
        b = np.zeros((1, N, K), dtype=np.float32)
        b[0, :, k * 32] = np.exp2(exps[:N, (k + 3) % (K // 32)])
        B, Bs = P().shp_mx4_quantize(torch.from_numpy(b).cuda())
        C = P().shp_mx4_matmul(A, As, B, Bs, dtype=torch.float32)
        np.testing.assert_array_equal(C.cpu().numpy(), a.astype(np.float64) @ b.astype(np.float64).transpose(0, 2, 1))


# many tiles: these run in tiles of 256 columns, the few of the sizes above in tiles of 128
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,M,N,K", [(5, 700, 1032, 1376), (40, 130, 264, 288), (38, 1, 8, 32), (1, 2500, 1800, 4192),
                                         (37, 256, 256, 96), (38, 256, 256, 96), (2, 100, 5000, 2080)])
def test_product_many_tiles(batch, M, N, K, dtype):
    A, As, a = operand(batch, M, K, 13)
    B, Bs, b = operand(batch, N, K, 14)
    C = P().shp_mx4_matmul(A, As, B, Bs, dtype=dtype)
    check_product(C, a, b)


def test_product_same_in_both_tile_widths():
    """A block alone (few tiles) and in a batch (many): the same bits."""
    A, As, _ = operand(40, 300, 1376, 15)
    B, Bs, _ = operand(40, 520, 1376, 16)
    for dtype in (torch.float32, torch.bfloat16):
        C = P().shp_mx4_matmul(A, As, B, Bs, dtype=dtype)
        for i in (0, 17, 39):
            one = P().shp_mx4_matmul(A[i:i + 1], As[i:i + 1], B[i:i + 1], Bs[i:i + 1], dtype=dtype)
            assert torch.equal(one[0], C[i])


def test_product_picks_every_scale_of_many_tiles():
    """test_product_picks_every_scale where tiles have 256 columns."""
    M, N, K = 2304, 1544, 288
    rows, blocks = torch.arange(M)[:, None], torch.arange(K // 32)[None, :]
    exps = ((rows * 7 + blocks * 5) % 23 - 11).double()
    for k in range(K // 32):
        a = torch.zeros(1, M, K, dtype=torch.float64)
        a[0, :, k * 32] = torch.exp2(exps[:, k])
        b = torch.zeros(1, N, K, dtype=torch.float64)
        b[0, :, k * 32] = torch.exp2(exps[:N, (k + 3) % (K // 32)])
        a, b = a.cuda(), b.cuda()
        A, As = P().shp_mx4_quantize(a.float())
        B, Bs = P().shp_mx4_quantize(b.float())
        C = P().shp_mx4_matmul(A, As, B, Bs, dtype=torch.float32)
        ref = a[0, :, k * 32, None] * b[0, None, :, k * 32]
        assert torch.equal(C[0].double(), ref)


def test_nan_block_reaches_its_row_alone():
    X = rand((1, 300, 256), 5, torch.float32)
    X[0, 77, 40] = float("nan")
    W, Ws, _ = operand(1, 264, 256, 6)
    A, As = P().shp_mx4_quantize(X)
    C = P().shp_mx4_matmul(A, As, W, Ws, dtype=torch.float32)
    nan = torch.isnan(C[0]).all(1)
    assert bool(nan[77]) and int(torch.isnan(C).any(2).sum()) == 1


def test_gradient_of_a_quantised_product():
    """Y = X W^T with W quantised along its columns; dX = dY W contracts over
    W's rows and reads the other orientation of the same matrix."""
    W = rand((1, 264, 512), 7, torch.float32)
    Q, S, Qt, St = P().shp_mx4_quantize(W, along="both")
    dY, dYs, dy = operand(1, 130, 264, 8)
    w = P().shp_mx4_dequantize(Qt, St, 264).double()  # W^T quantised along W's rows
    dX = P().shp_mx4_matmul(dY, dYs, Qt, St, dtype=torch.float32)
    check_product(dX, dy, torch.nn.functional.pad(w, (0, dy.shape[2] - 264)))


def test_streams_and_capture():
    X, W = rand((1, 500, 768), 9, torch.bfloat16), rand((1, 520, 768), 10, torch.bfloat16)
    B, Bs = P().shp_mx4_quantize(W)

    def linear():
        A, As = P().shp_mx4_quantize(X)
        return P().shp_mx4_matmul(A, As, B, Bs)

    ref = linear()
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            outs += [linear() for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = linear()
    X.copy_(rand((1, 500, 768), 11, torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, linear())


def test_large_offsets():
    """More than 2^32 elements: the last rows of a large batch."""
    batch, rows, cols = 70, 8192, 8192
    X = torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda")
    X[-1] = rand((rows, cols), 12, torch.bfloat16)
    Q, S, Qt, St = P().shp_mx4_quantize(X, along="both")
    one = P().shp_mx4_quantize(X[-1], along="both")
    for got, want in zip((Q, S, Qt, St), one):
        assert torch.equal(got[-1], want[0]) and not bool(got[:-1].any())
    del Qt, St
    assert torch.equal(P().shp_mx4_dequantize(Q, S, cols, dtype=torch.bfloat16)[-1],
                       P().shp_mx4_dequantize(one[0], one[1], cols, dtype=torch.bfloat16)[0])


def test_binding_refuses_wrong_tensors():
    p = P()
    A, As, _ = operand(1, 130, 256, 13)
    B, Bs, _ = operand(1, 136, 256, 14)
    with pytest.raises(ValueError):
        p.shp_mx4_matmul(A, As, B, Bs[:, :1])
    with pytest.raises(ValueError):
        p.shp_mx4_matmul(A, As, B[:, :, :64].contiguous(), Bs)
    with pytest.raises(ValueError):
        p.shp_mx4_matmul(A, As, B, Bs, dtype=torch.float16)
    with pytest.raises(ValueError):
        p.shp_mx4_dequantize(A, As, 300)
    with pytest.raises(ValueError):
        p.shp_mx4_quantize(torch.zeros(4, 4, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        p.shp_mx4_quantize(torch.zeros(64, 64, device="cuda"), along="x")
    with pytest.raises(RuntimeError):
        p.shp_mx4_quantize(torch.zeros(64, 62, device="cuda"))
