"""The binding's checks of devices for the expert-layer operators, with stand-ins for tensors of two GPUs and for the library
(no GPU needed)."""

import contextlib
import ctypes

import pytest
import torch

from token_permute_grouped_gb300 import binding


class On(torch.Tensor):
    """A tensor that says that it is on cuda:`index`."""

    is_cuda = True
    index = 0

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x1000


class Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 0x55


def on(index, *shape, dtype=torch.bfloat16):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.index = index
    return t


class Library:
    """Takes every call; notes its name, the current device and the stream."""

    def __init__(self, state):
        self.state, self.calls = state, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace_size"):
                ctypes.cast(args[-1], ctypes.POINTER(ctypes.c_size_t))[0] = 256
            else:
                self.calls.append((name, self.state["current"], args[-1]))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    state = {"current": 0}

    @contextlib.contextmanager
    def device(index):
        before, state["current"] = state["current"], index
        yield
        state["current"] = before

    library = Library(state)
    library.state = state
    monkeypatch.setattr(binding, "_lib", library)
    monkeypatch.setattr(binding, "_current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(binding, "_current_stream", lambda index: 0x100 + index)
    monkeypatch.setattr(binding, "_norm_backward_size", lambda *a: 256)
    real = binding._out
    monkeypatch.setattr(binding, "_out", lambda t, name, dtype, shape, like, stream:
                        on(like.get_device(), *shape, dtype=dtype) if t is None else real(t, name, dtype, shape, like, stream))
    return library


def plan(kind, index):
    """A plan whose workspace is on cuda:index."""
    p = kind.__new__(kind)
    p.desc = (binding.GatedDesc(2, 2, 4, 16, 8, 0, 0, 1, 1) if kind is binding.GatedPlan
              else binding.make_desc(2, 2, 4, 16, 8))
    p.dtype = torch.bfloat16
    p.workspace = on(index, 256, dtype=torch.uint8)
    return p


def calls(index):
    """name -> (the operands by name, a function of them and of stream)."""
    t = lambda *s, **k: on(index, *s, **k)
    counts = t(4, dtype=torch.int32)
    gated, gmm = plan(binding.GatedPlan, index), plan(binding.GmmBackwardPlan, index)
    f32 = dict(dtype=torch.float32)
    return {
        "a2av_rms_norm": (dict(x=t(4, 16), gamma=t(16), residual=t(4, 16)), binding.a2av_rms_norm),
        "a2av_rms_norm_backward": (dict(dy=t(4, 16), h=t(4, 16), gamma=t(16), rstd=t(4, **f32), dh=t(4, 16), dx=t(4, 16),
                                        dgamma=t(16, **f32), workspace=t(256, dtype=torch.uint8)),
                                   binding.a2av_rms_norm_backward),
        "a2av_glu_quant": (dict(gate_up=t(4, 16)), lambda gate_up, stream=None: binding.a2av_glu_quant(gate_up, qtype=None,
                                                                                                       stream=stream)),
        "a2av_gated_run": (dict(ataOut=t(4, 16), recvCounts=counts, gateWeight=t(2, 16, 8), upWeight=t(2, 16, 8), h=t(4, 8),
                                saved=t(2, 4, 8, **f32), permuteOut=t(4, 16)), gated.run),
        "a2av_gated_backward": (dict(dh=t(4, 8), permuteOut=t(4, 16), recvCounts=counts, gateWeight=t(2, 16, 8),
                                     upWeight=t(2, 16, 8), saved=t(2, 4, 8, **f32), dAtaOut=t(4, 16), dGate=t(2, 16, 8),
                                     dUp=t(2, 16, 8)), gated.backward),
        "a2av_gmm_backward": (dict(dY=t(4, 8), permuteOut=t(4, 16), recvCounts=counts, gmmWeight=t(2, 16, 8), dAtaOut=t(4, 16),
                                   dWeight=t(2, 16, 8)), gmm.run),
    }


NAMES = list(calls(0))


@pytest.mark.parametrize("name", NAMES)
def test_operands_of_another_device_are_refused(lib, name):
    operands, call = calls(0)[name]
    call(**operands)
    assert lib.calls == [(name, 0, 0x100)]
    for k in operands:
        if len(operands) == 1 or (k in ("x", "dy")):
            continue  # (the operand that names the device)
        moved = dict(operands)
        moved[k] = on(1, *operands[k].shape, dtype=operands[k].dtype)
        with pytest.raises(ValueError, match=f"{k} must be on cuda:0"):
            call(**moved)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("name", NAMES)
def test_the_call_is_made_on_the_tensors_device(lib, name):
    operands, call = calls(1)[name]
    call(**operands)
    assert lib.calls == [(name, 1, 0x101)] and lib.state["current"] == 0
    call(**operands, stream=Stream(1))
    assert lib.calls[-1] == (name, 1, 0x55)
    with pytest.raises(ValueError, match="stream must be of cuda:1"):
        call(**operands, stream=Stream(0))


def test_an_earlier_result_is_written_again_on_its_device(lib):
    x, gamma = on(1, 4, 16), on(1, 16)
    r = binding.a2av_rms_norm(x, gamma)
    assert binding.a2av_rms_norm(x, gamma, out=r) is r
    assert [c[1:] for c in lib.calls] == [(1, 0x101)] * 2
    with pytest.raises(ValueError, match="must be on cuda:0"):
        binding.a2av_rms_norm(on(0, 4, 16), on(0, 16), out=r)
