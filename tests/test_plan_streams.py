"""The plan's methods and the FP8 quantizers on a stream of the caller's: where their results come from."""
import contextlib

import pytest
import torch

import moe_megakernel_b200 as mk

T, H, I, E = 4, 128, 64, 8
BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


class Stream:
    cuda_stream = 5
    device = torch.device("cpu")


class Library:
    """Every C entry succeeds and does nothing."""
    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture
def plan(monkeypatch):
    p = mk.MoEPlan.__new__(mk.MoEPlan)
    p.__dict__.update(lib=Library(), device=torch.device("cpu"), T_max=T, H=H, I=I, E=E, k=2, n_shared=0, _plan=None)
    monkeypatch.setattr(mk, "load_library", Library)
    return p


def _t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


LAYER = [_t(T, H), _t(H, E), None, _t(E, H, I), _t(E, H, I), _t(E, I, H)]
FP8 = [_t(E, I, H, dtype=U8), _t(E, I, dtype=F32), _t(E, I, H, dtype=U8), _t(E, I, dtype=F32), _t(E, H, I, dtype=U8),
       _t(E, H, dtype=F32)]
DY = _t(T, H)


@pytest.mark.parametrize("call", [
    lambda p, s: p.forward(*LAYER, stream=s),
    lambda p, s: p.forward_fp8(*LAYER[:3], *FP8, stream=s),
    lambda p, s: p.backward(*LAYER, DY, stream=s),
    lambda p, s: mk.quantize_weights_fp8(LAYER[3], stream=s),
    lambda p, s: mk.quantize_x_fp8(DY, stream=s)], ids=["forward", "forward_fp8", "backward", "weights", "x"])
def test_results_are_allocated_on_the_stream_that_writes_them(call, plan, monkeypatch):
    inside, made, stream, empty = [], [], Stream(), torch.empty

    @contextlib.contextmanager
    def on(s):
        inside.append(s)
        yield
        inside.pop()

    def noted(*args, **kw):
        made.append(list(inside))
        return empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", noted)
    call(plan, stream)
    assert made and all(m == [stream] for m in made)
    assert not inside
