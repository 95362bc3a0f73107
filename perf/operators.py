"""Cases of the expert-grouped products and of the microscaled 4-bit format.

Four operators, each in its plain form (elementary torch operations in 32
bits) and as the library's calls:

  matmul    Y[t] = X[t] W_e(t): rows of X sorted by group, one weight block per
            group (the forward product of an expert layer; with W read
            transposed, the gradient of its input)
  wgrad     G[e] = A_e^T B_e (+ G[e]): the gradient of the weight blocks, in the
            [blocks][m][n] fp32 layout the optimizer's statistics take
  quantize  MXFP4 codes and scales of a batch of matrices, in blocks along the
            columns and (both) along the rows; returned as the values they
            stand for
  product   C[b] = A[b] B[b]^T of two MXFP4 operands

MXFP4: blocks of 32 values share a power-of-two scale 2^e (one byte, e + 127),
e = floor(log2 max|x|) - 2; an element is one of 0, .5, 1, 1.5, 2, 3, 4, 6 and
a sign, rounded to nearest (ties to the even code), two to a byte, low nibble
first.  Scales are stored in tiles of 128 rows x 4 blocks (512 bytes): row r,
block k of a tile at byte (r % 32) * 16 + (r / 32) * 4 + k.
"""
import math

import torch

own = False

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step: 16 rows spread over 64 expert blocks, most of them empty
        dict(name="matmul decode", op="matmul", T=16, E=64, K=1024, N=4096, trans=False, out="bf16", pad=0),
        # a prompt's rows over the same blocks: about 128 rows each
        dict(name="matmul prompt", op="matmul", T=8192, E=64, K=1024, N=4096, trans=False, out="bf16", pad=0),
        # the gradient of the input at training size, few large groups
        dict(name="matmul train dgrad", op="matmul", T=65536, E=16, K=4096, N=1024, trans=True, out="bf16", pad=0),
        # odd sizes, an fp32 result, rows behind the last group left as they were
        dict(name="matmul odd", op="matmul", T=1001, E=7, K=520, N=1032, trans=False, out="fp32", pad=23),
        # the 64 x 1024^2 weight blocks of the optimizer's batch: their gradients from 16384 rows
        dict(name="wgrad blocks", op="wgrad", T=16384, E=64, K=1024, N=1024, acc=False),
        # training size, accumulated over micro-batches
        dict(name="wgrad train", op="wgrad", T=65536, E=16, K=1024, N=4096, acc=True),
        # a short odd batch, some groups of a few rows or none
        dict(name="wgrad odd", op="wgrad", T=301, E=7, K=264, N=520, acc=False),
        # updated fp32 weight blocks to 4 bits, for the product (along columns) and its gradient (along rows)
        dict(name="quantize weights", op="quantize", rows=4096, cols=1024, batch=16, dtype="fp32", both=True),
        # a prompt's activations, one orientation
        dict(name="quantize rows", op="quantize", rows=8191, cols=4096, batch=1, dtype="bf16", both=False),
        # a large product of 4-bit operands
        dict(name="product large", op="product", M=8192, N=8192, K=4096, batch=1, out="bf16"),
        # a decoding step against 4-bit weights
        dict(name="product decode", op="product", M=16, N=4096, K=4096, batch=1, out="bf16"),
        # odd batched blocks, an fp32 result
        dict(name="product odd", op="product", M=300, N=1000, K=1376, batch=5, out="fp32"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v / step) * step if step > 1 else int(v)))


def draw(rng):
    op = rng.choice(["matmul", "wgrad", "quantize", "product"])
    if op in ("matmul", "wgrad"):
        K, N = _log(rng, 64, 4096, 8), _log(rng, 64, 4096, 8)
        E = _log(rng, 1, 96)
        T = _log(rng, 1, 65536)
        while T * K * N > 65536 * 4096 * 1024 or E * K * N > 64 * 4096 * 1024:
            T, E, K = max(1, T // 2), max(1, E // 2), max(64, K // 16 * 8)
        if op == "wgrad":
            return dict(op=op, T=T, E=E, K=K, N=N, acc=rng.random() < 0.5)
        return dict(op=op, T=T, E=E, K=K, N=N, trans=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]),
                    pad=rng.choice([0, 0, 1, 37]))
    if op == "quantize":
        dtype = rng.choice(["fp32", "bf16"])
        rows, cols = _log(rng, 1, 8192), _log(rng, 32, 8192, 8)
        batch = max(1, min(_log(rng, 1, 64), 16 * 4096 * 1024 // (rows * cols)))
        return dict(op=op, rows=rows, cols=cols, batch=batch, dtype=dtype, both=rng.random() < 0.5)
    M, N, K = _log(rng, 1, 8192), _log(rng, 64, 8192, 8), _log(rng, 32, 8192, 32)
    batch = _log(rng, 1, 32)
    while batch > 1 and batch * M * N * K > 2 ** 37:
        batch //= 2
    if M * N * K > 2 ** 38:
        K = 4096
    return dict(op=op, M=M, N=N, K=K, batch=batch, out=rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------ inputs
def _sizes(case, g):
    """Ragged group sizes that sum to T: popular and unpopular experts, some empty."""
    T, E = case["T"], case["E"]
    p = torch.rand(E, generator=g).pow(2) + 0.02
    counts = torch.bincount(torch.multinomial(p, T, replacement=True, generator=g), minlength=E)
    return [int(c) for c in counts]


def _values(shape, gen, dev):
    """Weights and activations: rows of unequal size, a few large entries, some zero blocks."""
    x = torch.randn(shape, generator=gen, device=dev)
    x *= torch.exp(torch.randn(shape[:-1] + (1,), generator=gen, device=dev))
    x *= 1 + 20 * (torch.rand(shape, generator=gen, device=dev) < 1e-3)
    x *= torch.rand(shape[:-1] + (1,), generator=gen, device=dev) > 0.01
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    randn = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    if op in ("matmul", "wgrad"):
        T, E, K, N = (case[k] for k in ("T", "E", "K", "N"))
        sizes = _sizes(case, host)
        edge = [0]
        for n in sizes:
            edge.append(edge[-1] + n)
        s["offsets"] = torch.tensor(edge, dtype=torch.int64).to(dev)
        s["cap"] = max(1, max(sizes))  # the largest group: the plain form's padded batch
        rows = T + case.get("pad", 0)
        s["X"] = randn(rows, K).to(torch.bfloat16)
        if op == "matmul":
            shape = (E, N, K) if case["trans"] else (E, K, N)
            s["W"] = (randn(*shape) / math.sqrt(K)).to(torch.bfloat16)
            s["Y"] = torch.zeros(rows, N, device=dev, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        else:
            s["dY"] = (randn(rows, N) * 0.1).to(torch.bfloat16)
            if case["acc"]:
                s["G"] = randn(E, K, N) * 0.1  # what earlier micro-batches left
    elif op == "quantize":
        x = _values((case["batch"], case["rows"], case["cols"]), gen, dev)
        s["X"] = x if case["dtype"] == "fp32" else x.to(torch.bfloat16)
    else:
        for name, rows in (("A", case["M"]), ("B", case["N"])):
            q, e = _plain_codes(_values((case["batch"], rows, case["K"]), gen, dev))
            s[name], s[name + "s"] = q[..., 0::2] | (q[..., 1::2] << 4), _tile(e)
    return s


def _tile(e):
    """[batch][rows][blocks] scale bytes -> [batch][rows/128][blocks/4][512] tiles, zero-padded."""
    b, r, k = e.shape
    rt, kt = (r + 127) // 128, (k + 3) // 4
    p = torch.zeros(b, rt * 128, kt * 4, dtype=torch.uint8, device=e.device)
    p[:, :r, :k] = e
    return p.view(b, rt, 4, 32, kt, 4).permute(0, 1, 4, 3, 2, 5).reshape(b, rt, kt, 512)


def _untile(t, rows, blocks):
    b, rt, kt, _ = t.shape
    return t.view(b, rt, kt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(b, rt * 128, kt * 4)[:, :rows, :blocks]


# -------------------------------------------------------------- plain forms
def _plain_codes(x):
    """Codes (one per byte) and scale bytes of the last axis, padded with zeros to whole blocks."""
    x = x.float()
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 32))
    blk = x.unflatten(-1, (-1, 32))
    amax = blk.abs().amax(-1)
    e = torch.frexp(amax).exponent - 3  # frexp's mantissa is in [1/2, 1): floor(log2) is one less
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    y = torch.ldexp(blk, -e[..., None])
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = (torch.round(a / step) * step).clamp(max=6.0)  # round: half to even
    code = torch.where(v < 2, v * 2, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _decode(code, e):
    """fp32 values of codes (one per byte) under scale bytes."""
    lut = torch.tensor(_GRID + tuple(-v for v in _GRID), device=code.device)
    v = lut[code.long()].unflatten(-1, (-1, 32))
    return torch.ldexp(v, (e.to(torch.int32) - 127)[..., None]).flatten(-2)


def _operand(q, tiles):
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    return _decode(code, _untile(tiles, q.shape[1], code.shape[-1] // 32))


def _padded(x, off, cap):
    """The groups of x as a batch [E][cap][.], zero behind a group's rows."""
    at = off[:-1, None] + torch.arange(cap, device=x.device)
    ok = at < off[1:, None]
    return torch.where(ok[..., None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0), at, ok


def _plain(s):
    op = s["op"]
    if op == "matmul":
        xp, at, ok = _padded(s["X"], s["offsets"], s["cap"])
        w = s["W"].float()
        y = torch.matmul(xp, w.transpose(1, 2) if s["trans"] else w)
        s["Y"][at[ok]] = y[ok].to(s["Y"].dtype)
        return s["Y"]
    if op == "wgrad":
        a, _, _ = _padded(s["X"], s["offsets"], s["cap"])
        b, _, _ = _padded(s["dY"], s["offsets"], s["cap"])
        g = torch.matmul(a.transpose(1, 2), b)
        return s["G"].add_(g) if s["acc"] else g
    if op == "quantize":
        def values(x):
            return _decode(*_plain_codes(x))[..., : x.shape[-1]].to(x.dtype)
        return (values(s["X"]), values(s["X"].transpose(1, 2))) if s["both"] else values(s["X"])
    c = torch.matmul(_operand(s["A"], s["As"]), _operand(s["B"], s["Bs"]).transpose(1, 2))
    return c.to(torch.bfloat16) if s["out"] == "bf16" else c


def run(s):
    if not own:
        return _plain(s)
    from second_order_optimizer_shampoo_b200 import prism
    op = s["op"]
    if op == "matmul":
        return prism.shp_grouped_matmul(s["X"], s["offsets"], s["W"], w_trans=s["trans"], out=s["Y"])
    if op == "wgrad":
        if s["acc"]:
            return prism.shp_grouped_wgrad(s["X"], s["dY"], s["offsets"], out=s["G"], accumulate=True)
        return prism.shp_grouped_wgrad(s["X"], s["dY"], s["offsets"])
    if op == "quantize":
        X = s["X"]
        if s["both"]:
            Q, S, Qt, St = prism.shp_mx4_quantize(X, along="both")
            return (prism.shp_mx4_dequantize(Q, S, X.shape[2], dtype=X.dtype),
                    prism.shp_mx4_dequantize(Qt, St, X.shape[1], dtype=X.dtype))
        Q, S = prism.shp_mx4_quantize(X)
        return prism.shp_mx4_dequantize(Q, S, X.shape[2], dtype=X.dtype)
    return prism.shp_mx4_matmul(s["A"], s["As"], s["B"], s["Bs"],
                                dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)


# --------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "matmul":
        T, E, K, N = (case[k] for k in ("T", "E", "K", "N"))
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * T * K + 2 * min(T, E) * K * N + out * T * N + 8 * (E + 1), "flops": 2 * T * K * N}
    if op == "wgrad":
        T, E, K, N = (case[k] for k in ("T", "E", "K", "N"))
        return {"bytes": 2 * T * (K + N) + (8 if case["acc"] else 4) * E * K * N, "flops": 2 * T * K * N}
    if op == "quantize":
        n = case["batch"] * case["rows"] * case["cols"]
        size = 4 if case["dtype"] == "fp32" else 2
        each = n * 2 * (1 / 2 + 1 / 32) + n * size  # codes and scales written and read, values written
        return {"bytes": n * size + each * (2 if case["both"] else 1), "flops": 4 * n}
    M, N, K, b = (case[k] for k in ("M", "N", "K", "batch"))
    out = 2 if case["out"] == "bf16" else 4
    return {"bytes": b * ((M + N) * K * (1 / 2 + 1 / 32) + out * M * N), "flops": 2 * b * M * N * K}


# -------------------------------------------------------------- in 64 bits
def _exact_codes(x):
    """Values of the MXFP4 form of the last axis, by comparison with the midpoints of the grid."""
    n = x.shape[-1]
    x = x.double()
    full = x.new_zeros(x.shape[:-1] + (-(-n // 32) * 32,))
    full[..., :n] = x
    blk = full.reshape(x.shape[:-1] + (-1, 32))
    top = blk.abs().max(-1, keepdim=True).values
    e = torch.floor(torch.log2(top))
    e = torch.where(torch.exp2(e) > top, e - 1, e)  # log2 next to a power of two
    e = torch.where(torch.exp2(e + 1) <= top, e + 1, e)
    scale = torch.exp2(torch.where(top > 0, e - 2, torch.zeros_like(e)).clamp(-127, 127))
    a = blk.abs() / scale
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    v = torch.zeros_like(a)
    for i in range(7):
        mid = (grid[i] + grid[i + 1]) / 2
        v = torch.where((a > mid) if i % 2 == 0 else (a >= mid), grid[i + 1], v)
    return (torch.sign(blk) * v * scale).reshape(full.shape)[..., :n]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("matmul", "wgrad"):
        edge = s["offsets"].tolist()
        X = s["X"]
        if op == "matmul":
            Y = torch.zeros(s["Y"].shape, dtype=torch.float64, device=X.device)
            for e in range(case["E"]):
                a, b = edge[e], edge[e + 1]
                w = s["W"][e].double()
                Y[a:b] = X[a:b].double() @ (w.t() if case["trans"] else w)
            return Y
        G = s["G"].double() if case["acc"] else torch.zeros(case["E"], case["K"], case["N"], dtype=torch.float64, device=X.device)
        for e in range(case["E"]):
            a, b = edge[e], edge[e + 1]
            G[e] += X[a:b].double().t() @ s["dY"][a:b].double()
        return G
    if op == "quantize":
        rows = _exact_codes(s["X"])
        return (rows, _exact_codes(s["X"].transpose(1, 2).contiguous())) if case["both"] else rows

    def operand(q, tiles):  # by the layout's own formula
        b, r, half = q.shape
        grid = torch.tensor(_GRID, dtype=torch.float64, device=q.device)
        v = torch.empty(b, r, 2 * half, dtype=torch.float64, device=q.device)
        for i, nib in enumerate((q & 15, q >> 4)):
            v[..., i::2] = grid[(nib & 7).long()] * (1 - 2 * (nib >> 3).double())
        row = torch.arange(r, device=q.device)[:, None]
        k = torch.arange(2 * half // 32, device=q.device)[None, :]
        byte = tiles[:, row // 128, k // 4, (row % 32) * 16 + (row % 128) // 32 * 4 + k % 4]
        return v * torch.exp2(byte.double() - 127).repeat_interleave(32, -1)

    return operand(s["A"], s["As"]) @ operand(s["B"], s["Bs"]).transpose(1, 2)
