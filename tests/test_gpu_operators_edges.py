"""The operators around the layer at the edges of what they take, against 64-bit formulas."""
import math

import pytest
import torch

import moe_megakernel_b200 as mk
from tests.test_gpu_operators import (BF, HF, U, act64, close, gradient, offsets_of, ortho64, ortho_close, rand,
                                      slope64, spans)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,dtype", [
    ((64, 1032, 520), BF), ((2400, 264, 136), BF), ((2400, 264, 135), BF), ((1200, 264, 136), torch.float32),
    ((2400, 135, 264), torch.float32)])
def test_orthogonalize_batches_with_several_pieces_to_a_warp(shape, dtype):
    """A warp of the scaling pass turns two to six 32 x 32 pieces one after the other through the same
    shared memory: every matrix of a large batch stays as near its 64-bit form as a matrix by itself."""
    G = gradient(*shape, seed=131, dtype=dtype)
    out = mk.orthogonalize(G)
    for at in range(0, shape[0], 400):
        ortho_close(out[at:at + 400], G[at:at + 400])


FAR = [0.0, 1e-30, 0.25, 0.75, 2.0, 7.5, 20.0, 100.0, 3000.0, 6e4, 1e9, 1.5e13, 4e13, 1e16, 8e19, 1e25, 1e30, 3.3e38]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_of_far_preactivations(act, dtype):
    """Up to the type's largest value a slope is a number: 0 or 1 where the activation has gone flat or
    straight, and no NaN gets from one pre-activation into a row of dx or a column of dW. Tolerance: the
    rounding, and 1e-5 for the fp32 evaluation (an exponential good to 2 + 1.17 |v| units of 2^-23, whose
    weight in a slope, |z v'| e^-|v|, is below 1.2)."""
    z = torch.tensor([s * v for v in FAR if dtype == BF or v < 65504 for s in (1, -1)], device="cuda", dtype=dtype)
    z = torch.cat([z, z.new_zeros(-len(z) % 8)])
    N = len(z)
    x, W = torch.zeros(1, 8, dtype=dtype, device="cuda"), torch.ones(8, N, dtype=dtype, device="cuda")
    x[0, 3] = 1
    dy = torch.ones(1, N, dtype=dtype, device="cuda")
    g = mk.linear_backward(dy, x, W, preact=z[None], activation=act, bias_grad=True)
    ref = slope64(z.double(), act)
    for name, got in (("dbias", g["dbias"]), ("dW", g["dW"][3])):
        off = (got.double() - ref).abs()
        assert (off <= U[dtype] * ref.abs() + 1e-5).all(), (name, z[~(off <= U[dtype] * ref.abs() + 1e-5)])
    assert (g["dW"][:3] == 0).all() and (g["dW"][4:] == 0).all()
    assert ((g["dx"].double() - ref.sum()).abs() <= 2 * U[dtype] * ref.abs().sum() + 1e-5 * N).all()


@pytest.mark.parametrize("T", [1, 700])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_of_far_preactivations(act, T):
    """The same for the values, through both kernels, and NaN stays NaN. Tolerance as above: an
    activation's own weight |z| e^-|v| is below 1.2 as well."""
    z = torch.tensor([s * v for v in FAR for s in (1, -1)] + [float("nan")] * 4, device="cuda", dtype=BF)
    W = torch.zeros(8, len(z), dtype=BF, device="cuda")
    x = torch.zeros(T, 8, dtype=BF, device="cuda")
    x[:, 5] = 1
    b = z.clone()          # z = 0 + b: exact
    y, kept = mk.linear(x, W, bias=b, activation=act, save_preact=True)
    ref = act64(z.double(), act)
    number = ~z.isnan()
    assert torch.equal(kept[:, number], z[number].expand(T, -1)) and kept[:, ~number].isnan().all()
    assert y[:, ~number].isnan().all()
    assert ((y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5)[:, number].all()


def tail64(z, act):
    """An activation, without the cancellation of 1 + tanh(u) at the far negative end: z / (1 + e^(-2u))."""
    if act != "gelu_tanh":
        return act64(z, act)
    return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [1, 600])
def test_activations_keep_their_small_values(act, T, dtype):
    """Every z of the type in -12 .. 6 (fp16: every eighth): the value and the slope are off by the rounding
    and 2^-15 of themselves, however small they are. 2^-15 = 3e-5: the exponential is good to 2 + 1.17 |v|
    units of 2^-23 (|v| <= 72: 1e-5 at most) and its argument is rounded three times
    (3 |v| 2^-24: 1.3e-5 at most). A slope's two terms cancel around z = -1, so its error counts against
    their magnitudes; fp16 values below 2^-14 are rounded in steps of 2^-24."""
    i = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16)
    z = i.view(dtype)
    z = z[(z >= (-12 if act != "gelu_tanh" else -9)) & (z <= 6) & (z.abs() >= 2.0 ** -13)]
    z = z[::8 if dtype == HF else 1]
    z = z[:len(z) // 8 * 8].contiguous()
    W, x = torch.zeros(8, len(z), dtype=dtype, device="cuda"), torch.zeros(T, 8, dtype=dtype, device="cuda")
    ones = torch.ones(T, len(z), dtype=dtype, device="cuda")
    tiny = 2.0 ** -25 if dtype == HF else 0.0
    y = mk.linear(x, W, bias=z, activation=act)
    z64 = z.double().requires_grad_()
    value = tail64(z64, act)
    slope, = torch.autograd.grad(value.sum(), z64)
    value = value.detach()
    assert ((y.double() - value).abs() <= (U[dtype] + 2.0 ** -15) * value.abs() + tiny).all()
    x[0, 0] = 1            # dW[0] is the first row's dz
    got = mk.linear_backward(ones, x, W, preact=z.expand(T, -1).contiguous(), activation=act)["dW"][0].double()
    parts = (value / z.double()).abs()    # q, or Phi
    parts = parts + (slope - parts).abs()
    assert ((got - slope).abs() <= U[dtype] * slope.abs() * 1.01 + 2.0 ** -15 * parts + 2 * tiny).all()


@pytest.mark.parametrize("T", [1, 600])
def test_silu_keeps_its_smallest_values(T):
    """silu and its slope down to z = -90, where they are near bf16's smallest normal number: the rounding
    (below that number half a step, 2^-134), and 2^-15 for an exponential good to 2 + 1.17 * 90 units of 2^-23."""
    z = torch.linspace(-90, -12, 1000, device="cuda").to(BF)
    W, x = torch.zeros(8, len(z), dtype=BF, device="cuda"), torch.zeros(T, 8, dtype=BF, device="cuda")
    y = mk.linear(x, W, bias=z, activation="silu")
    ref = act64(z.double(), "silu")
    assert ((y.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -15) * ref.abs() + 2.0 ** -134).all()
    x[0, 0] = 1
    got = mk.linear_backward(torch.ones(T, len(z), dtype=BF, device="cuda"), x, W, preact=z.expand(T, -1).contiguous(),
                             activation="silu")["dW"][0].double()
    ref = slope64(z.double(), "silu")
    assert ((got - ref).abs() <= (2.0 ** -8 + 2.0 ** -14) * ref.abs() + 2.0 ** -133).all()


def _stream_calls():
    x, W = rand(300, 512, seed=141), rand(512, 264, seed=142, std=0.05)
    Wg, off, dy = rand(4, 512, 264, seed=143, std=0.05), offsets_of([100, 0, 150, 50]), rand(300, 264, seed=144)
    G = gradient(512, 264, seed=145)
    return {
        "grouped_matmul": ((300, 264), lambda s: mk.grouped_matmul(x, Wg, off, stream=s)),
        "grouped_matmul_wgrad": ((4, 512, 264), lambda s: mk.grouped_matmul_wgrad(x, dy, off, stream=s)),
        "linear": ((300, 264), lambda s: mk.linear(x, W, stream=s)),
        "linear_backward": ((512, 264), lambda s: mk.linear_backward(dy, x, W, input_grad=False, stream=s)["dW"]),
        "orthogonalize": ((512, 264), lambda s: mk.orthogonalize(G, stream=s)),
    }


@pytest.mark.parametrize("name", ["grouped_matmul", "grouped_matmul_wgrad", "linear", "linear_backward", "orthogonalize"])
def test_results_on_an_explicit_stream_take_no_other_streams_memory(name):
    """A result written on a side stream neither lands in a block that the current stream's queued work
    still reads, nor, dropped at once, is its block handed to the current stream while the kernel runs."""
    shape, call = _stream_calls()[name]
    side = torch.cuda.Stream()
    ref = call(None)
    torch.cuda.synchronize()
    a, b = (torch.full(shape, v, dtype=BF, device="cuda") for v in (7.0, 0.0))
    torch.cuda._sleep(40_000_000)      # some 20 ms
    b.copy_(a)
    del a
    y = call(side)
    torch.cuda.synchronize()
    assert (b == 7).all() and torch.equal(y, ref)
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    call(side)                         # dropped
    c = torch.full(shape, 7.0, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    assert (c == 7).all()


def _long_reduction(rows):
    """x, dy [rows, 8], zeros but for some rows at the ends, in the middle and around them."""
    g = torch.Generator().manual_seed(151)
    at = torch.cat([torch.tensor([0, 1, 63, 64, rows // 2, rows - 65, rows - 2, rows - 1]),
                    torch.randint(0, rows, (200,), generator=g)]).unique().cuda()
    x, dy = (torch.zeros(rows, 8, dtype=BF, device="cuda") for _ in range(2))
    x[at], dy[at] = rand(len(at), 8, seed=152), rand(len(at), 8, seed=153)
    a, b = x[at].double(), dy[at].double()
    return x, dy, a.T @ b, a.abs().T @ b.abs(), len(at)


def test_reductions_of_most_of_a_billion_rows():
    """One tile's reduction takes seconds, longer than any wait inside an ordinary call. Zero rows add
    nothing, so the sum has the roundings of the other rows alone."""
    rows = (3 << 28) + 37         # some 3.3 s in one tile, 6e9 cycles
    x, dy, ref, S, n = _long_reduction(rows)
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    dW = mk.grouped_matmul_wgrad(x, dy, off, error_word=err[:1])
    torch.cuda.synchronize()
    dense = mk.linear_backward(dy, x, dW[0], input_grad=False, error_word=err[1:])["dW"]
    assert err.tolist() == [0, 0]
    close(dW[0], ref, S, n)
    close(dense, ref, S, n)


def test_calls_queued_behind_seconds_of_work():
    """The kernels of the calls that follow set out early, on the SMs that a one-tile reduction leaves idle,
    and stand there for seconds: their waits count from its end. (No error words: zeroing one comes between.)"""
    rows = (3 << 28) + 37
    x, dy, ref, S, n = _long_reduction(rows)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    few = off.clamp(max=300)
    torch.cuda.synchronize()
    dW = mk.grouped_matmul_wgrad(x, dy, off)
    up = mk.orthogonalize(dW[0])
    other = mk.grouped_matmul(x[:300], dW, few)
    close(dW[0], ref, S, n)
    ortho_close(up, dW[0])
    a, w = x[:300].double(), dW[0].double()
    close(other, a @ w, a.abs() @ w.abs(), 8)


def test_ragged_tails_of_many_groups_give_the_same_bits():
    """Every group ends inside a step of 16 rows, with infinities behind it: zeros that the follower of a
    pair writes over the neighbour's rows are there before the leader multiplies them, in every run."""
    g = torch.Generator().manual_seed(161)
    counts = [int(c) for c in torch.randint(1, 400, (96,), generator=g)]
    counts = [c + 1 if c % 16 == 0 else c for c in counts]
    off, rows = offsets_of(counts), sum(counts)
    x, dy = rand(rows, 264, seed=162), rand(rows, 328, seed=163)
    last = torch.tensor([hi - 1 for _, _, hi in spans(off)[1::2]], device="cuda")   # of every other group
    x[last], dy[last] = float("inf"), float("nan")
    first = mk.grouped_matmul_wgrad(x, dy, off)
    for e, lo, hi in spans(off)[0::2]:
        a, b = x[lo:hi].double(), dy[lo:hi].double()
        close(first[e], a.T @ b, a.abs().T @ b.abs(), hi - lo, f"group {e}")
    for _ in range(30):
        assert torch.equal(mk.grouped_matmul_wgrad(x, dy, off)[0::2], first[0::2])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("shape", [(192, 320), (320, 192), (40, 61), (2, 300, 520)])
@pytest.mark.parametrize("spread", [1e6, 1e7])
def test_orthogonalize_brings_small_rows_up(spread, shape, dtype):
    """All rows but one (columns of a tall matrix) a millionth of the others' size and less, and a dozen
    steps, which bring them to size: relative Frobenius error as of ortho_close for 12 steps, sqrt(36) * 8e-4
    and 1.6e-3 in quadrature, 5.2e-3."""
    g = torch.Generator(device="cuda").manual_seed(171)
    G = torch.randn(shape, generator=g, device="cuda") * 1e-3
    if shape[-2] > shape[-1]:
        G[..., 3] *= spread
    else:
        G[..., 3, :] *= spread
    G = G.to(dtype)
    out, ref = mk.orthogonalize(G, steps=12), ortho64(G, steps=12)
    size = ref.flatten(-2).norm(dim=-1)
    err = (out.double() - ref).flatten(-2).norm(dim=-1)
    assert (err <= 5.2e-3 * size).all(), (err / size).max()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_orthogonalize_gradients_far_below_eps(dtype):
    """A norm of 1e-12 beside an eps of 1e-7: X starts at 1e-5 and the steps bring it up. Tolerance as above."""
    G = gradient(48, 80, seed=172)
    G = (G * (1e-12 / G.norm())).to(dtype)
    out, ref = mk.orthogonalize(G, steps=12), ortho64(G, steps=12)
    assert (out.double() - ref).norm() <= 5.2e-3 * ref.norm()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("coeffs", [mk.QUINTIC, (1.0, 0.5, 0.25), (1.5, 0.5, 0.0), (2.0, 0.0, 0.0)])
def test_orthogonalize_makes_a_matrix_with_an_infinity_nan_whatever_the_coefficients(coeffs, dtype):
    G = gradient(4, 40, 72, seed=173).abs().to(dtype)
    G[1, 7, 9] = float("inf")
    G[2, 39, 71] = float("nan")
    out = mk.orthogonalize(G, steps=2, coeffs=coeffs)
    assert out[1].isnan().all() and out[2].isnan().all()
    assert out[0].isfinite().all() and out[3].isfinite().all()
    one = torch.full((1, 1), float("inf"), dtype=dtype, device="cuda")
    assert mk.orthogonalize(one, steps=1, coeffs=coeffs).isnan().all()


def test_captured_calls_with_error_words_and_a_forked_stream():
    """A capture that holds zeroed error words between the kernels, and one whose calls run on a second
    stream beside the first, replay to the plain calls' bits."""
    x, W, off = rand(300, 512, seed=181), rand(4, 512, 264, seed=182, std=0.05), offsets_of([100, 0, 150, 50])
    dy, z, G, W1 = rand(300, 264, seed=183), rand(300, 264, seed=184), gradient(3, 140, 100, seed=185), W[1].contiguous()
    err = torch.full((6,), 9, dtype=torch.int32, device="cuda")

    def work():
        b = mk.linear_backward(dy, x, W1, preact=z, activation="gelu", bias_grad=True, error_word=err[0:1])
        return [mk.grouped_matmul(x, W, off, error_word=err[1:2]),
                mk.grouped_matmul_wgrad(x, dy, off, error_word=err[2:3]),
                mk.linear(x, W1, activation="silu", error_word=err[3:4]), mk.linear(x[:3], W1, error_word=err[4:5]),
                b["dx"], b["dW"], b["dbias"], mk.orthogonalize(G, error_word=err[5:6])]

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    assert err.tolist() == [9] * 6
    for _ in range(3):
        graph.replay()
    assert err.tolist() == [0] * 6
    ref = work()
    assert all(torch.equal(a, b) for a, b in zip(ref, outs))
    side, forked = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(forked):
        side.wait_stream(torch.cuda.current_stream())
        y, u = mk.linear(x[:3], W1, stream=side), mk.orthogonalize(G, stream=side)
        v = mk.grouped_matmul(x, W, off)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        forked.replay()
    torch.cuda.synchronize()
    assert torch.equal(v, ref[0]) and torch.equal(y, ref[3]) and torch.equal(u, ref[7])


def test_orthogonalize_in_place():
    for shape in ((130, 90), (3, 90, 130)):
        G = gradient(*shape, seed=191, dtype=BF)
        ref = mk.orthogonalize(G)
        assert mk.orthogonalize(G, out=G) is G and torch.equal(G, ref)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("m,n,spread", [(20, 30, 1e3), (30, 20, 1e3), (40, 60, 1e4), (200, 300, 1e4)])
def test_orthogonalize_of_one_direction_far_above_the_others(m, n, spread, dtype):
    """The other directions, among few of which a rounding of the large one's entries spreads, keep the
    accuracy of ortho_close. (A bf16 gradient has rounded them itself; the 64-bit form starts from that.)"""
    g = torch.Generator(device="cuda").manual_seed(201)
    u, v = (torch.linalg.qr(torch.randn(k, k, device="cuda", dtype=torch.float64, generator=g))[0] for k in (m, n))
    s = torch.full((min(m, n),), 1 / spread, device="cuda", dtype=torch.float64)
    s[0] = 1.0
    G = ((u[:, :len(s)] * s) @ v[:len(s)]).to(dtype)
    ortho_close(mk.orthogonalize(G), G)
