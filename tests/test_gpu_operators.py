"""The operators around the layer against plain 64-bit formulas.

Tolerances. A stored value is rounded once: at most u |y| with u = eps / 2 of its type (bf16
2^-8, fp16 2^-11). The fp32 accumulation of K exact products adds at most K 2^-23 S, where S is
the sum of the products' magnitudes (each of the K additions drops at most one unit in the last
place of a partial sum, which S bounds). `close` checks u |y| + (K + 4) 2^-23 S for every entry;
activations and residuals are 1-Lipschitz up to 1.13 and cost a few more fp32 roundings.
"""
import math

import pytest
import torch

import moe_megakernel_b200 as mk

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}


def rand(*shape, seed, dtype=BF, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def close(got, ref, S, K, what="", slope=1.0):
    """|got - ref| <= u |ref| + slope (K + 4) 2^-23 S, entry by entry."""
    assert got.shape == ref.shape
    u = U[got.dtype]
    # below the smallest normal number a rounding is absolute (fp16 2^-25)
    tol = u * ref.abs() + slope * (K + 4) * 2.0 ** -23 * S * (1 + u) + (2.0 ** -25 if got.dtype == HF else 0.0)
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} entries off, first at {bad.nonzero()[0].tolist()}, " \
                          f"worst {(err / tol).max().item():.3g} of the tolerance"


def offsets_of(counts, start=0):
    return torch.tensor([start] + [start + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32,
                        device="cuda")


def spans(offsets):
    o = offsets.tolist()
    return list(zip(range(len(o) - 1), o[:-1], o[1:]))


RAGGED = [0, 1, 31, 32, 33, 0, 64, 100, 255, 256, 257, 513, 2, 0]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts,K,N", [
    (RAGGED, 192, 264), (RAGGED, 72, 520), ([1], 8, 8), ([3, 0, 5], 128, 256), ([1] * 40, 200, 328),
    ([0, 0, 0, 700], 1000, 128), ([20] * 16, 64, 64), ([50] * 9, 328, 96),
    ([300, 0, 150, 420, 178], 2000, 352)])
def test_grouped_matmul(counts, K, N, transpose, dtype):
    off = offsets_of(counts)
    rows = sum(counts)
    x = rand(rows, K, seed=1, dtype=dtype)
    W = rand(len(counts), *((N, K) if transpose else (K, N)), seed=2, dtype=dtype, std=K ** -0.5)
    err = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    y = mk.grouped_matmul(x, W, off, transpose=transpose, error_word=err)
    assert err.item() == 0
    for e, lo, hi in spans(off):
        w = W[e].double().T if transpose else W[e].double()
        close(y[lo:hi], x[lo:hi].double() @ w, x[lo:hi].double().abs() @ w.abs(), K, f"group {e}")


def test_grouped_rows_outside_the_groups_stay_and_do_not_spread():
    """Rows before the first and behind the last group keep their bits; NaN there, in other groups
    and in other groups' weights reaches no group's output."""
    counts, K, N = [40, 3, 0, 77], 136, 272
    off = offsets_of(counts, start=5)
    rows = 5 + sum(counts) + 30
    x, W = rand(rows, K, seed=3), rand(4, K, N, seed=4, std=K ** -0.5)
    x[:5] = float("nan")
    x[5 + sum(counts):] = float("inf")
    x[45:48] = float("nan")     # group 1
    W[1] = float("inf")
    W[2] = float("nan")         # an empty group's weights
    y = torch.full((rows, N), 3.25, dtype=BF, device="cuda")
    mk.grouped_matmul(x, W, off, y=y)
    assert (y[:5] == 3.25).all() and (y[5 + sum(counts):] == 3.25).all()
    assert y[45:48].isnan().all()
    for e, lo, hi in [spans(off)[0], spans(off)[3]]:
        close(y[lo:hi], x[lo:hi].double() @ W[e].double(), x[lo:hi].double().abs() @ W[e].double().abs(), K)


def test_grouped_strided_rows_and_many_groups():
    """Row pitches beyond the row, and the most groups a call takes, most of them empty."""
    K, N, groups = 72, 88, 1024
    g = torch.Generator().manual_seed(0)
    counts = [int(c) if i % 5 == 0 else 0 for i, c in enumerate(torch.randint(0, 40, (groups,), generator=g))]
    counts[groups - 1] = 41
    off, rows = offsets_of(counts), sum(counts)
    xs, ys = rand(rows, K + 16, seed=17), torch.full((rows, N + 24), 3.25, dtype=BF, device="cuda")
    x, y = xs[:, 8:8 + K], ys[:, 16:16 + N]
    W = rand(groups, K, N, seed=18, std=K ** -0.5)
    mk.grouped_matmul(x, W, off, y=y)
    dW = mk.grouped_matmul_wgrad(x, y, off)
    assert (ys[:, :16] == 3.25).all() and (ys[:, 16 + N:] == 3.25).all()
    for e, lo, hi in spans(off):
        a, b = x[lo:hi].double(), y[lo:hi].double()
        close(y[lo:hi], a @ W[e].double(), a.abs() @ W[e].double().abs(), K, f"group {e}")
        close(dW[e], a.T @ b, a.abs().T @ b.abs(), hi - lo, f"dW {e}")


@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [-1, 2, 4, 9], [0, 4, 6, 99]])
def test_grouped_bad_offsets_are_recorded_and_skipped(bad):
    K, N = 64, 64
    x, W = rand(9, K, seed=5), rand(3, K, N, seed=6, std=K ** -0.5)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((9, N), 3.25, dtype=BF, device="cuda")
    mk.grouped_matmul(x, W, off, y=y, error_word=err)
    assert err.item() == 2
    dW = mk.grouped_matmul_wgrad(x, y, off, error_word=err)
    assert err.item() == 2
    for e, (lo, hi) in enumerate(zip(bad[:-1], bad[1:])):
        if not 0 <= lo <= hi <= 9:
            assert (dW[e] == 0).all()
    err.fill_(9)
    mk.grouped_matmul(x, W, offsets_of([3, 3, 3]), y=y, error_word=err)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,K,N", [
    (RAGGED, 192, 264), (RAGGED, 72, 520), ([1], 8, 8), ([0], 64, 64), ([15, 16, 17, 63, 65, 130], 328, 136),
    ([0, 0, 1500, 0], 256, 256), ([7] * 30, 96, 40)])
def test_wgrad(counts, K, N, dtype):
    off = offsets_of(counts, start=3)
    rows = 3 + sum(counts) + 2
    x, dy = rand(rows, K, seed=7, dtype=dtype), rand(rows, N, seed=8, dtype=dtype, std=0.3)
    for t in (x, dy):
        t[:3] = float("nan")
        t[rows - 2:] = float("inf")
    dW = mk.grouped_matmul_wgrad(x, dy, off, dW=torch.full((len(counts), K, N), 9.0, dtype=dtype, device="cuda"))
    for e, lo, hi in spans(off):
        a, b = x[lo:hi].double(), dy[lo:hi].double()
        close(dW[e], a.T @ b, a.abs().T @ b.abs(), hi - lo, f"group {e}")


def test_wgrad_other_groups_infinities_stay_theirs():
    counts, K, N = [17, 20, 100], 128, 128
    off = offsets_of(counts)
    x, dy = rand(137, K, seed=9), rand(137, N, seed=10)
    x[17:37] = float("inf")
    dy[17:37] = float("nan")
    dW = mk.grouped_matmul_wgrad(x, dy, off)
    assert dW[1].isnan().all()
    for e in (0, 2):
        lo, hi = spans(off)[e][1:]
        a, b = x[lo:hi].double(), dy[lo:hi].double()
        close(dW[e], a.T @ b, a.abs().T @ b.abs(), hi - lo)


def test_grouped_gradients_against_differences():
    """d/dx and d/dW of L = sum(c * y) against central differences of the 64-bit product."""
    counts, K, N = [5, 0, 12], 64, 72
    off = offsets_of(counts)
    x, W, c = rand(17, K, seed=11), rand(3, K, N, seed=12, std=0.125), rand(17, N, seed=13)
    dx = mk.grouped_matmul(c, W, off, transpose=True)
    dW = mk.grouped_matmul_wgrad(x, c, off)

    def loss(xd, Wd):
        return sum((c[lo:hi].double() * (xd[lo:hi] @ Wd[e])).sum() for e, lo, hi in spans(off))

    g = torch.Generator(device="cuda").manual_seed(14)
    for of in ("x", "W"):
        t = x.double() if of == "x" else W.double()
        d = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 0.5    # the loss is linear in each: any step is exact
        plus, minus = ((loss(t + s * h * d, W.double()) if of == "x" else loss(x.double(), t + s * h * d))
                       for s in (1, -1))
        grad = (dx if of == "x" else dW).double()
        # each entry of the gradient is off by at most 2^-8 of itself
        tol = 2.0 ** -8 * (grad * d).abs().sum() * 1.01
        assert abs((plus - minus) / (2 * h) - (grad * d).sum()) <= tol


def test_zero_rows():
    off = offsets_of([0, 0])
    x, W = rand(0, 64, seed=1), rand(2, 64, 32, seed=2)
    assert mk.grouped_matmul(x, W, off).shape == (0, 32)
    assert (mk.grouped_matmul_wgrad(x, rand(0, 32, seed=3), off) == 0).all()
    assert mk.linear(x, W[0]).shape == (0, 32)
    g = mk.linear_backward(rand(0, 32, seed=3), x, W[0], bias_grad=True)
    assert g["dx"].shape == (0, 64) and (g["dW"] == 0).all() and (g["dbias"] == 0).all()
    assert mk.orthogonalize(torch.zeros(0, 5, 7, device="cuda")).shape == (0, 5, 7)


def act64(z, act):
    return {None: lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: 0.5 * z * torch.erfc(-z / math.sqrt(2)),
            "gelu_tanh": lambda: torch.nn.functional.gelu(z, approximate="tanh")}[act]()


def slope64(z, act):
    if act is None:
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    z = z.clone().requires_grad_()
    act64(z, act).sum().backward()
    return z.grad


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,K,N,act,bias,res,save", [
    (1, 64, 128, None, False, False, False), (1, 4096, 512, "silu", True, False, False),
    (7, 1000, 264, "gelu", True, True, True), (16, 512, 1032, "relu", False, True, False),
    (33, 2056, 96, "gelu_tanh", True, False, True), (64, 136, 4104, None, True, True, True),
    (65, 64, 64, "silu", False, False, True), (128, 328, 640, "gelu", True, True, True),
    (129, 8, 8, "relu", True, True, True), (300, 584, 776, "silu", True, True, False),
    (37, 8192, 264, "gelu", True, True, True), (200, 4096, 512, "silu", True, True, True),
    (500, 6000, 136, None, True, True, True), (31, 320, 40000, "relu", True, False, False),
    (2100, 136, 1288, "gelu", True, True, True), (384, 6000, 2056, "silu", True, True, True),
    (512, 2048, 1000, None, False, True, False), (700, 3000, 264, "gelu", True, False, True),
    (1031, 256, 520, "gelu", True, False, True)])
def test_linear(T, K, N, act, bias, res, save, dtype):
    x, W = rand(T, K, seed=21, dtype=dtype), rand(K, N, seed=22, dtype=dtype, std=K ** -0.5)
    b = rand(N, seed=23, dtype=dtype) if bias else None
    r = rand(T, N, seed=24, dtype=dtype) if res else None
    got = mk.linear(x, W, bias=b, activation=act, residual=r, save_preact=save)
    y, z = got if save else (got, None)
    zr = x.double() @ W.double()
    S = x.double().abs() @ W.double().abs()
    if bias:
        zr, S = zr + b.double(), S + b.double().abs()
    if save:
        close(z, zr, S, K, "preact")
    ref = act64(zr, act)
    if res:
        ref, S = ref + r.double(), S + r.double().abs()
    close(y, ref, S + zr.abs(), K, "y", slope=1.13)


def test_linear_onto_the_residual_itself_and_strided_rows():
    T, K, N = 77, 192, 272
    big = rand(T, K + 24, seed=31)
    x = big[:, 8:8 + K]                       # rows 216 elements apart, 16-byte aligned
    W = rand(K, N, seed=32, std=K ** -0.5)
    store = rand(T, N + 8, seed=33)
    before = store.clone()
    y = store[:, :N]
    ref = x.double() @ W.double() + y.double()
    S = x.double().abs() @ W.double().abs() + y.double().abs()
    mk.linear(x, W, residual=y, y=y)
    close(y, ref, S, K)
    assert torch.equal(store[:, N:], before[:, N:])
    with pytest.raises(ValueError):
        mk.linear(rand(T, K + 4, seed=1)[:, :K], W)          # rows 196 elements apart
    with pytest.raises(mk.MoEError):
        mk.linear(rand(T, K + 8, seed=1)[:, 4:4 + K], W)     # rows start 8 bytes off


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,K,N,act,bias", [
    (1, 64, 128, "silu", True), (5, 8, 8, None, True), (37, 520, 264, "gelu", True), (128, 136, 1032, "relu", False),
    (200, 256, 256, "gelu_tanh", True), (1031, 328, 520, "silu", True), (4100, 64, 72, None, True),
    (64, 256, 4096, "gelu", True), (150, 520, 6000, "silu", False), (3812, 104, 776, None, False),
    (1598, 664, 256, "silu", True), (2051, 24, 136, "relu", True), (777, 200, 96, "gelu", False), (5000, 300 * 2, 520, "silu", True),
    (384, 1000, 6000, "gelu", True)])
def test_linear_backward(T, K, N, act, bias, dtype):
    x, W = rand(T, K, seed=41, dtype=dtype), rand(K, N, seed=42, dtype=dtype, std=K ** -0.5)
    dy = rand(T, N, seed=43, dtype=dtype, std=0.2)
    z = rand(T, N, seed=44, dtype=dtype) if act else None
    g = mk.linear_backward(dy, x, W, preact=z, activation=act, bias_grad=bias)
    dz = dy.double() * (slope64(z.double(), act) if act else 1.0)
    # dz enters the products rounded once: one more u of each product's magnitudes
    u = U[dtype] if act else 0.0
    a, b, w = dz.abs(), x.double().abs(), W.double().abs()
    tiny = 2.0 ** -25 if dtype == HF and act else 0.0   # fp16 rounding of a subnormal dz
    for got, ref, S, n, side in ((g["dx"], dz @ W.double().T, a @ w.T, N, w.sum(1)[None, :]),
                                 (g["dW"], x.double().T @ dz, b.T @ a, T, b.sum(0)[:, None])):
        tol = U[dtype] * ref.abs() + (1.01 * u + (n + 16) * 2.0 ** -23) * S + tiny * side + 2.0 ** -25
        err = (got.double() - ref).abs()
        assert (err <= tol).all(), (err / tol).max()
    if bias:
        close(g["dbias"], dz.sum(0), a.sum(0), T + 16, "dbias")
    only = mk.linear_backward(dy, x, W, preact=z, activation=act, input_grad=False, weight_grad=True)
    assert only["dx"] is None and only["dbias"] is None and torch.equal(only["dW"], g["dW"])


def test_linear_backward_against_differences():
    T, K, N = 9, 64, 40
    x, W, b = rand(T, K, seed=51), rand(K, N, seed=52, std=0.125), rand(N, seed=53, std=0.1)
    c = rand(T, N, seed=54)
    _, z = mk.linear(x, W, bias=b, activation="gelu", save_preact=True)
    g = mk.linear_backward(c, x, W, preact=z, activation="gelu", bias_grad=True)
    gen = torch.Generator(device="cuda").manual_seed(55)
    dirs = [torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) for t in (x, W, b)]

    def loss(s, i):
        xs, ws, bs = (t.double() + (s * d if j == i else 0) for j, (t, d) in enumerate(zip((x, W, b), dirs)))
        return (c.double() * act64(xs @ ws + bs, "gelu")).sum()

    for i, name in enumerate(("dx", "dW", "dbias")):
        h = 1e-4
        want = (loss(h, i) - loss(-h, i)) / (2 * h)
        terms = g[name].double() * dirs[i]
        # z, dz and the result are each rounded to bf16 (2^-8; the slope's own slope is below 0.8 and
        # |z| below 4, so z's rounding moves a slope by at most 0.0125); every entry by its own sum
        dzabs = c.double().abs()
        mag = {"dx": dzabs @ W.double().abs().T, "dW": x.double().abs().T @ dzabs, "dbias": dzabs.sum(0)}[name]
        tol = (2.0 ** -8 * terms.abs() + (0.0125 + 2.0 ** -8 * 1.13) * mag * dirs[i].abs()).sum()
        assert abs(want - terms.sum()) <= tol


def ortho64(G, steps=5, coeffs=mk.QUINTIC, eps=1e-7):
    X = G.double()
    X = X / (X.flatten(-2).norm(dim=-1)[..., None, None] + eps)
    rows = coeffs if isinstance(coeffs[0], (list, tuple)) else [coeffs] * steps
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.mT
    for a, b, c in rows:
        A = X @ X.mT
        X = a * X + (b * A + c * A @ A) @ X
    return X.mT if tall else X


def ortho_close(got, G, **kw):
    """Relative Frobenius error of every matrix <= 5e-3: the bf16 output's rounding is 0.41 * 2^-8 = 1.6e-3
    (root mean square over the mantissa), and each of the steps' 3 fp16 roundings adds independently
    at most about 4 * 0.41 * 2^-11 = 8e-4 (4: the largest gain |b s + 2 c s^2| + |b s + c s^2| of a step),
    in quadrature sqrt(15) * 8e-4 = 3.1e-3; together 3.5e-3. No entry is off by more than that of a
    whole singular direction."""
    assert got.dtype == BF and got.shape == G.shape
    ref = ortho64(G, **kw)
    err = (got.double() - ref).flatten(-2).norm(dim=-1)
    assert (err <= 5e-3 * ref.flatten(-2).norm(dim=-1)).all(), (err / ref.flatten(-2).norm(dim=-1)).max()


def gradient(*shape, seed, dtype=torch.float32, rank=4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    *b, m, n = shape
    u, v = torch.randn(*b, m, rank, generator=g, device="cuda"), torch.randn(*b, rank, n, generator=g, device="cuda")
    return ((u @ v) * 1e-3 + 2e-4 * torch.randn(shape, generator=g, device="cuda")).to(dtype)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (5, 3), (33, 64), (64, 33), (129, 250), (250, 129),
                                   (256, 256), (3, 130, 70), (5, 40, 300), (2, 513, 257), (300, 1031), (1000, 520),
                                   (40, 300, 520), (40, 520, 300), (90, 130, 140), (7, 2375, 30), (300, 20, 33), (58, 28, 1835)])
def test_orthogonalize(shape, dtype):
    G = gradient(*shape, seed=61, dtype=dtype, rank=min(4, *shape[-2:]))
    ortho_close(mk.orthogonalize(G), G)


def test_orthogonalize_spreads_of_singular_values():
    """A gradient dominated by one direction a thousand times the others: the small directions keep their
    relative accuracy, because a X is added from the 22-bit X."""
    u = torch.linalg.qr(torch.randn(200, 200, device="cuda", dtype=torch.float64,
                                    generator=torch.Generator(device="cuda").manual_seed(71)))[0]
    v = torch.linalg.qr(torch.randn(300, 300, device="cuda", dtype=torch.float64,
                                    generator=torch.Generator(device="cuda").manual_seed(72)))[0]
    s = torch.full((200,), 1e-3, device="cuda", dtype=torch.float64)
    s[0] = 1.0
    G = ((u * s) @ v[:200]).float()
    ortho_close(mk.orthogonalize(G), G)


def test_orthogonalize_scales_and_special_values():
    G = gradient(6, 48, 80, seed=73)
    G[0] *= 1e30
    G[1] *= 1e-25        # norm near 1e-27, far below eps: the result vanishes
    G[2] = 0
    G[3, 5, 7] = float("inf")
    G[4, 0, 0] = float("nan")
    out = mk.orthogonalize(G)
    ortho_close(out[[0, 5]], G[[0, 5]])
    assert (out[1].abs() < 1e-6).all() and (out[2] == 0).all()
    assert out[3].isnan().all() and out[4].isnan().all()


def test_orthogonalize_steps_coefficients_and_pitches():
    big = gradient(4, 70, 120, seed=74)
    G = big[1:3, 3:60, 5:98]
    sched = [(3.5, -6.0, 3.2), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)]
    store = torch.full((2, 60, 101), 7.0, dtype=BF, device="cuda")
    out = store[:, 1:58, 3:96]
    got = mk.orthogonalize(G, steps=3, coeffs=sched, out=out)
    assert got.data_ptr() == out.data_ptr()
    ortho_close(got, G, coeffs=sched)
    assert (store[:, 0] == 7).all() and (store[:, 58:] == 7).all()
    assert (store[:, :, :3] == 7).all() and (store[:, :, 96:] == 7).all()
    tall = gradient(3, 130, 80, seed=76)[:2, 5:112, 7:72]
    for dtype in (torch.float32, BF):
        src = tall.to(dtype) if dtype == BF else tall
        wide = torch.full((2, 110, 72), 7.0, dtype=BF, device="cuda")
        mk.orthogonalize(src, out=wide[:, 2:109, 4:69])
        ortho_close(wide[:, 2:109, 4:69], src)
        assert (wide[:, :2] == 7).all() and (wide[:, 109:] == 7).all()
        assert (wide[:, :, :4] == 7).all() and (wide[:, :, 69:] == 7).all()
    one = gradient(40, 90, seed=75)
    ortho_close(mk.orthogonalize(one, steps=1, coeffs=(1.5, -0.5, 0.0)), one, steps=1, coeffs=(1.5, -0.5, 0.0))


def test_same_bits_every_time():
    x, W = rand(300, 512, seed=81), rand(512, 256, seed=82, std=0.05)
    off = offsets_of([100, 0, 150, 50])
    Wg = rand(4, 512, 256, seed=83, std=0.05)
    G = gradient(2, 130, 90, seed=84)
    dy, z = rand(300, 256, seed=85), rand(300, 256, seed=86)
    def all_of():
        b = mk.linear_backward(dy, x, W, preact=z, activation="silu", bias_grad=True)
        return [mk.linear(x, W, activation="gelu"), mk.linear(x[:5], W), mk.grouped_matmul(x, Wg, off),
                mk.grouped_matmul_wgrad(x, dy, off), b["dx"], b["dW"], b["dbias"], mk.orthogonalize(G)]
    first = all_of()
    for _ in range(3):
        for a, b in zip(first, all_of()):
            assert torch.equal(a, b)


def test_two_streams_and_captured_graphs():
    """Calls on two streams at once and two graphs replayed at once give the plain calls' bits."""
    off = offsets_of([100, 3, 150, 47])
    x, W = rand(300, 512, seed=91), rand(4, 512, 264, seed=92, std=0.05)
    dy, G = rand(300, 264, seed=93), gradient(3, 140, 100, seed=94)
    W1, z = W[0].contiguous(), rand(300, 264, seed=95)

    def work(stream=None):
        b = mk.linear_backward(dy, x, W1, preact=z, activation="gelu", bias_grad=True, stream=stream)
        return [mk.grouped_matmul(x, W, off, stream=stream), mk.grouped_matmul_wgrad(x, dy, off, stream=stream),
                mk.linear(x, W1, activation="silu", stream=stream), mk.linear(x[:3], W1, stream=stream), b["dx"],
                b["dW"], b["dbias"], mk.orthogonalize(G, stream=stream)]

    ref = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = work(s)
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(ref, g))
    # a stream given explicitly while another is current
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = work(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, g))
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(work())
        graphs.append(gr)
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for g in outs:
        assert all(torch.equal(a, b) for a, b in zip(ref, g))


def test_offsets_past_32_bits():
    """A weight set and an activation whose element offsets pass 2^31."""
    K, N, groups = 4096, 8192, 70                      # 70 x 33.5 M = 2.35e9 elements
    W = torch.zeros(groups, K, N, dtype=BF, device="cuda")
    W[groups - 1] = rand(K, N, seed=111, std=K ** -0.5)
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[groups] = 50
    x = rand(50, K, seed=112)
    y = mk.grouped_matmul(x, W, off)
    ref, S = x.double() @ W[-1].double(), x.double().abs() @ W[-1].double().abs()
    close(y, ref, S, K)
    dW = mk.grouped_matmul_wgrad(x, y, off, dW=W)
    assert (dW[:groups - 1] == 0).all()
    close(dW[-1], x.double().T @ y.double(), x.double().abs().T @ y.double().abs(), 50)
    del W, dW
    T, K, N = 280_000, 64, 8192                        # 2.29e9 outputs
    x, W = rand(T, K, seed=113), rand(K, N, seed=114, std=0.125)
    y = mk.linear(x, W)
    tail = slice(T - 300, T)
    close(y[tail], x[tail].double() @ W.double(), x[tail].double().abs() @ W.double().abs(), K)


def test_orthogonalized_steps_of_a_training_loop():
    """Two steps of a dense layer trained with orthogonalised updates, all captured in one graph: every
    replay moves the weights as the same calls outside the graph do."""
    T, K, N = 200, 128, 264
    x, t = rand(T, K, seed=121), rand(T, N, seed=122)
    W0, b0 = rand(K, N, seed=123, std=K ** -0.5), rand(N, seed=124, std=0.1)

    def step(W, b):
        y, z = mk.linear(x, W, bias=b, activation="silu", save_preact=True)
        g = mk.linear_backward(y - t, x, W, preact=z, activation="silu", bias_grad=True)
        W.sub_(mk.orthogonalize(g["dW"]), alpha=0.02)
        b.sub_(g["dbias"], alpha=1e-3)

    Wa, ba = W0.clone(), b0.clone()
    for _ in range(3):
        step(Wa, ba)
        step(Wa, ba)
    Wg, bg = W0.clone(), b0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(Wg, bg)
        step(Wg, bg)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Wa, Wg) and torch.equal(ba, bg)
    assert not torch.equal(Wg, W0)


def test_layer_from_its_parts():
    """The operators together, on the routing of a MoEPlan: the layer's forward and weight gradients from
    grouped products, and the update of its gradients. Tolerances as the layer's own parity tests
    (relative Frobenius 1e-2) plus one more bf16 rounding per step."""
    T, H, I, E, k = 300, 256, 128, 8, 2
    x, Wg = rand(T, H, seed=101), rand(H, E, seed=102, std=H ** -0.5)
    W1, W3 = (rand(E, H, I, seed=s, std=H ** -0.5) for s in (103, 104))
    W2, dy = rand(E, I, H, seed=105, std=I ** -0.5), rand(T, H, seed=106)
    plan = mk.MoEPlan(T, H, I, E, k, backward=True)
    y = plan.forward(x, Wg, None, W1, W3, W2)
    plan.check()
    r = plan.routing(T)
    P, off = int(r["num_padded"]), r["expert_offset"].clone()
    tok, pos = r["slot_token"][:P].long(), r["slot_topk"][:P].long()
    real = tok >= 0
    xs = torch.where(real[:, None], x[tok.clamp_min(0)], torch.zeros((), dtype=BF, device="cuda"))
    w = torch.where(real, r["topk_w"][tok.clamp_min(0), pos.clamp_min(0)], 0.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    g, u = (mk.grouped_matmul(xs, W, off, error_word=err) for W in (W1, W3))
    a = (torch.nn.functional.silu(g.float()) * u.float()).to(BF)
    o = mk.grouped_matmul(a, W2, off)
    mine = torch.zeros(T, H, device="cuda").index_add_(0, tok[real], (w[:, None] * o.float())[real])
    assert (mine - y.float()).norm() <= 1.5e-2 * y.float().norm()
    grads = plan.backward(x, Wg, None, W1, W3, W2, dy)
    plan.check()
    dys = torch.where(real[:, None], dy[tok.clamp_min(0)], torch.zeros((), dtype=BF, device="cuda"))
    dys = (w[:, None] * dys.float()).to(BF)
    dW2 = mk.grouped_matmul_wgrad(a, dys, off)
    da = mk.grouped_matmul(dys, W2, off, transpose=True).float()
    sg = torch.sigmoid(g.float())
    dg = (da * u.float() * sg * (1 + g.float() * (1 - sg))).to(BF)
    dW1 = mk.grouped_matmul_wgrad(xs, dg, off)
    for got, ref in ((dW2, grads["dW2"]), (dW1, grads["dW1"])):
        assert (got.float() - ref.float()).norm() <= 1.5e-2 * ref.float().norm()
    assert err.item() == 0
    ortho_close(mk.orthogonalize(grads["dW1"]), grads["dW1"])
    ortho_close(mk.orthogonalize(grads["dW2"]), grads["dW2"])
    # the residual stream through a dense projection
    Wd = rand(H, H, seed=107, std=H ** -0.5)
    h = mk.linear(y, Wd, residual=x)
    close(h, y.double() @ Wd.double() + x.double(), y.double().abs() @ Wd.double().abs() + x.double().abs(), H)
