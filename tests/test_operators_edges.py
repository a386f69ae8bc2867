"""The operators around the layer, what can be seen of them without a GPU."""
import contextlib

import pytest
import torch

import moe_megakernel_b200 as mk
from moe_megakernel_b200 import operators
from tests.test_operators import BF, _off, _z


@pytest.fixture(scope="module", autouse=True)
def lib():
    from moe_megakernel_b200 import build, load_library
    build.build()
    return load_library()


class Stream:
    """Stands for a stream of the tensors' device (here the host)."""
    cuda_stream = 5
    device = torch.device("cpu")


CALLS = {
    "grouped_matmul": lambda s: mk.grouped_matmul(_z(4, 64), _z(2, 64, 32), _off(0, 2, 4), stream=s),
    "grouped_matmul_wgrad": lambda s: mk.grouped_matmul_wgrad(_z(4, 64), _z(4, 32), _off(0, 2, 4), stream=s),
    "linear": lambda s: mk.linear(_z(4, 64), _z(64, 32), save_preact=True, stream=s),
    "linear_backward": lambda s: mk.linear_backward(_z(4, 32), _z(4, 64), _z(64, 32), preact=_z(4, 32), activation="silu",
                                                    bias_grad=True, stream=s),
    "orthogonalize": lambda s: mk.orthogonalize(_z(4, 6), stream=s),
}


@pytest.fixture
def calls(monkeypatch):
    """The C calls are noted down instead of made; argument checks that need a GPU pass."""
    made = []
    monkeypatch.setattr(operators, "_cuda", lambda t, name: None)
    monkeypatch.setattr(operators, "_call", lambda name, device, *args: made.append((name, args)))
    return made


@pytest.fixture
def allocations(monkeypatch):
    """For every tensor made from here on, the streams that were current."""
    inside, made = [], []

    @contextlib.contextmanager
    def on(s):
        inside.append(s)
        yield
        inside.pop()

    def noted(f):
        def g(*args, **kw):
            made.append(list(inside))
            return f(*args, **kw)
        return g

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.Tensor, "new_empty", noted(torch.Tensor.new_empty))
    monkeypatch.setattr(torch, "empty", noted(torch.empty))
    return made


@pytest.mark.parametrize("name", CALLS)
def test_results_are_allocated_on_the_stream_that_writes_them(name, calls, allocations):
    """A block of another stream's pool may still be read by work queued there."""
    stream = Stream()
    CALLS[name](stream)
    assert allocations and all(made == [stream] for made in allocations)
    assert calls[0][0] == "moe_" + name and calls[0][1][-1] == 5


def test_streams_of_other_devices_are_refused(calls):
    class Other(Stream):
        device = torch.device("cuda", 1)
    for call in CALLS.values():
        with pytest.raises(ValueError, match="stream"):
            call(Other())
    assert not calls


META = torch.device("meta")
BIG = 2 ** 32 + 8      # 8 in its lower 32 bits


def _m(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device=META)


class MetaStream(Stream):
    device = META


@pytest.mark.parametrize("call", [
    lambda s: mk.grouped_matmul(_m(BIG, 8), _m(2, 8, 16), _m(3, dtype=torch.int32), stream=s),
    lambda s: mk.grouped_matmul(_m(4, BIG), _m(2, BIG, 16), _m(3, dtype=torch.int32), stream=s),
    lambda s: mk.grouped_matmul(_m(4, 8), _m(2, 8, BIG), _m(3, dtype=torch.int32), stream=s),
    lambda s: mk.grouped_matmul(_m(4, 8), _m(2, BIG, 8), _m(3, dtype=torch.int32), transpose=True, stream=s),
    lambda s: mk.grouped_matmul(_m(4, 8), _m(BIG, 8, 16), _m(BIG + 1, dtype=torch.int32), stream=s),
    lambda s: mk.grouped_matmul_wgrad(_m(BIG, 8), _m(BIG, 16), _m(3, dtype=torch.int32), stream=s),
    lambda s: mk.grouped_matmul_wgrad(_m(4, BIG), _m(4, 16), _m(3, dtype=torch.int32), stream=s),
    lambda s: mk.grouped_matmul_wgrad(_m(4, 8), _m(4, BIG), _m(3, dtype=torch.int32), stream=s),
    lambda s: mk.grouped_matmul_wgrad(_m(4, 8), _m(4, 8), _m(BIG + 1, dtype=torch.int32), stream=s),
    lambda s: mk.linear(_m(BIG, 8), _m(8, 16), stream=s),
    lambda s: mk.linear(_m(4, BIG), _m(BIG, 16), stream=s),
    lambda s: mk.linear(_m(4, 8), _m(8, BIG), stream=s),
    lambda s: mk.linear_backward(_m(BIG, 16), _m(BIG, 8), _m(8, 16), stream=s),
    lambda s: mk.linear_backward(_m(4, BIG), _m(4, 8), _m(8, BIG), stream=s),
    lambda s: mk.linear_backward(_m(4, 16), _m(4, BIG), _m(BIG, 16), stream=s),
    lambda s: mk.orthogonalize(_m(BIG, 4, 4), stream=s),
    lambda s: mk.orthogonalize(_m(BIG, 4), stream=s),
    lambda s: mk.orthogonalize(_m(4, BIG), stream=s),
    lambda s: mk.orthogonalize(_m(4, 4), steps=65, stream=s),
    lambda s: mk.quantize_x_fp8(_m(BIG, 8), stream=s),
    lambda s: mk.quantize_weights_fp8(_m(BIG, 64, 64), stream=s),
    lambda s: mk.MoEPlan(2 ** 32 + 64, 128, 256, 8, 2, device="cuda:0")])
def test_extents_past_32_bits_are_refused(call, calls):
    """Not taken for their lower 32 bits, which the C entry would find nothing wrong with."""
    with pytest.raises(mk.MoEError, match="MOE_ERR_UNSUPPORTED_SHAPE"):
        call(MetaStream())
    assert not calls


@pytest.mark.parametrize("call", [
    lambda x, W, s: mk.grouped_matmul(x, W[None], _off(0, 8), y=x, stream=s),
    lambda x, W, s: mk.grouped_matmul(x, W[None], _off(0, 8), y=W, stream=s),
    lambda x, W, s: mk.grouped_matmul_wgrad(x, W, _off(0, 8), dW=x[None], stream=s),
    lambda x, W, s: mk.grouped_matmul_wgrad(x, W, _off(0, 8), dW=W[None], stream=s),
    lambda x, W, s: mk.linear(x, W, y=x, stream=s),
    lambda x, W, s: mk.linear(x, W, y=W, stream=s),
    lambda x, W, s: mk.linear(x, W, preact=x, stream=s),
    lambda x, W, s: mk.linear(x, W, residual=_z(8, 8), preact=W, stream=s),
    lambda x, W, s: (lambda r: mk.linear(x, W, residual=r, preact=r, stream=s))(_z(8, 8)),
    lambda x, W, s: (lambda r: mk.linear(x, W, y=r, preact=r, stream=s))(_z(8, 8)),
    lambda x, W, s: (lambda r: mk.linear(x, W, y=r[:8], residual=r.view(8, 16)[:, :8], stream=s))(_z(16, 8))])
def test_results_on_top_of_inputs_are_refused(call, calls):
    with pytest.raises(ValueError, match="overlaps"):
        call(_z(8, 8), _z(8, 8), Stream())
    assert not calls


def test_results_that_may_share_memory(calls):
    x, W, r = _z(8, 8), _z(8, 8), _z(8, 8)
    assert mk.linear(x, W, residual=r, y=r, stream=Stream()) is r
    assert mk.orthogonalize(x, out=x, stream=Stream()) is x
    assert len(calls) == 2
