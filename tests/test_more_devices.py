"""The binding's checks of devices for the layer norm, the product with a scale per 128 and the few-token expert layer, with
stand-ins for tensors of two GPUs and for the library (no GPU needed)."""

import pytest
import torch

import test_ffn_devices as D
from test_ffn_devices import lib, on  # noqa: F401
from token_permute_grouped_gb300 import binding


def f32(index, *shape):
    return on(index, *shape, dtype=torch.float32)


def u8(index, *shape):
    return on(index, *shape, dtype=torch.uint8)


def counts(index, n):
    return on(index, n, dtype=torch.int32)


def g128_plan(index):
    plan = binding.G128Plan(2, 2, 8, 256, 64, device="cpu")
    plan.workspace = u8(index, 1024)
    return plan


def moe_plan(index):
    plan = binding.MoePlan(2, 4, 2, 64, 64, device="cpu")
    plan.workspace = u8(index, 1024)
    return plan


def norm_args(i):
    return dict(x=on(i, 4, 256), gamma=on(i, 256), beta=on(i, 256), residual=on(i, 4, 256))


def back_args(i):
    return dict(dy=on(i, 4, 256), h=on(i, 4, 256), gamma=on(i, 256), mean=f32(i, 4), rstd=f32(i, 4), dh=on(i, 4, 256),
                dx=on(i, 4, 256), dgamma=f32(i, 256), dbeta=f32(i, 256), workspace=u8(i, 1 << 16))


def g128_args(i):
    return dict(ataOut_q=u8(i, 8, 256), ataOut_s=f32(i, 8, 2), recvCounts=counts(i, 4), gmmWeight_q=u8(i, 2, 64, 256),
                gmmWeight_s=f32(i, 2, 1, 2), gmmY=on(i, 8, 64))


def moe_args(i):
    return dict(x=on(i, 2, 64), router=on(i, 4, 64), gate=on(i, 4, 64, 64), up=on(i, 4, 64, 64), down=on(i, 4, 64, 64),
                bias=f32(i, 4), residual=on(i, 2, 64),
                out=binding.MoeOut(on(i, 2, 64), on(i, 2, 2, dtype=torch.int32), f32(i, 2, 2)))


def calls(i, **replaced):
    """name -> (entry point, call with tensors of cuda:i, some replaced)."""
    with_ = lambda a: {**a, **{k: v for k, v in replaced.items() if k in a}}
    return {
        "layer_norm": ("a2av_layer_norm", norm_args(i), lambda a: binding.a2av_layer_norm(
            **a, qtype=None, out=binding.LayerNormOut(on(i, 4, 256), on(i, 4, 256), None, None, None, None))),
        "layer_norm_backward": ("a2av_layer_norm_backward", back_args(i), lambda a: binding.a2av_layer_norm_backward(**a)),
        "g128": ("a2av_gmm_g128_run", g128_args(i), lambda a: g128_plan(i).run(**a)),
        "moe": ("a2av_moe_run", moe_args(i), lambda a: moe_plan(i).run(**a)),
    }


NAMES = ["layer_norm", "layer_norm_backward", "g128", "moe"]


@pytest.mark.parametrize("name", NAMES)
def test_the_operands_device_is_current_during_the_call(lib, name):  # noqa: F811
    entry, args, call = calls(1)[name]
    call(args)
    made = [c for c in lib.calls if c[0] == entry]
    assert len(made) == 1 and made[0][1] == 1  # on cuda:1, which was not the current device


# (The norms' first operand says which device it is.)
OPERANDS = [(n, k) for n in NAMES for i, k in enumerate(calls(0)[n][1]) if k != "out" and (i > 0 or n in ("g128", "moe"))]


@pytest.mark.parametrize("name,which", OPERANDS)
def test_tensors_of_another_device_are_refused(lib, name, which):  # noqa: F811
    entry, args, call = calls(0)[name]
    moved = D.on(1, *args[which].shape, dtype=args[which].dtype)
    with pytest.raises(ValueError, match="must be on cuda:0"):
        call({**args, which: moved})
    assert not [c for c in lib.calls if c[0] == entry]


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(lib, name):  # noqa: F811
    entry, args, call = calls(0)[name]
    fn = {"layer_norm": lambda s: binding.a2av_layer_norm(args["x"], args["gamma"], stream=s, out=binding.LayerNormOut(
              None, on(0, 4, 256), None, None, None, None)),
          "layer_norm_backward": lambda s: binding.a2av_layer_norm_backward(**args, stream=s),
          "g128": lambda s: g128_plan(0).run(**args, stream=s), "moe": lambda s: moe_plan(0).run(**args, stream=s)}[name]
    with pytest.raises(ValueError, match="stream must be of cuda:0"):
        fn(D.Stream(1))
    assert not [c for c in lib.calls if c[0] == entry]
