"""The training-step binding's argument checks, on the host: tensors of another
device than the handle's are refused before the library is called."""
import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import Checkpoint, FgError, TrainingOps, _lib


class OnDevice:
    """A tensor on device `device`, as far as the checks look at it."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.float32, device=0):
        self.t, self.device = torch.empty(shape, dtype=dtype), device
        self.shape, self.dtype = self.t.shape, dtype
        self.stride, self.data_ptr = self.t.stride, self.t.data_ptr
        self.is_contiguous, self.numel = self.t.is_contiguous, self.t.numel

    def get_device(self):
        return self.device


class Calls:
    """A library that notes which functions are called."""

    def __init__(self):
        self.seen = []

    def __getattr__(self, name):
        return lambda *a: self.seen.append(name) or _lib.FG_OK


@pytest.fixture
def ops():
    o = TrainingOps.__new__(TrainingOps)
    o.lib, o.h, o.device = Calls(), None, 0
    return o


def arguments():
    """Every call with its tensors, by name."""
    def x(d=0): return OnDevice((4, 64), device=d)
    def b(d=0): return OnDevice((4, 64), torch.bfloat16, d)
    def v(d=0): return OnDevice((64,), device=d)
    def s(d=0): return OnDevice((4,), device=d)
    def ck(d=0): return Checkpoint(4, 64, OnDevice((4 * 132,), torch.uint8, d))
    def t(d=0): return OnDevice((4,), torch.int64, d)
    def top(d=0): return OnDevice((4, 2), device=d)
    def ids(d=0): return OnDevice((4, 2), torch.int32, d)
    def dw(d=0): return OnDevice((64, 64), device=d)
    return {
        "layer_norm": (x, v, v, x, s, s, None, ck),
        "layer_norm_backward": (x, x, v, s, s, x, v, v),
        "checkpoint_save": (x, ck),
        "checkpoint_load": (ck, x),
        "activation_backward": ("tanh", x, ck, x),
        "weight_grad": (ck, b, dw, v, v, v),
        "token_logprobs": (x, t, s, s, s, top, ids),
        "token_logprobs_backward": (x, t, s, s, s, s, x),
    }


CASES = [(name, i) for name, args in arguments().items() for i, a in enumerate(args) if callable(a)]
CASES.append(("layer_norm_backward", "checkpoint"))


def made(name, wrong):
    args = list(arguments()[name])
    if wrong == "checkpoint":
        args[1], wrong = arguments()["checkpoint_save"][1], 1
    return [1e-5 if a is None else a(int(i == wrong)) if callable(a) else a for i, a in enumerate(args)]


@pytest.mark.parametrize("name, wrong", CASES)
def test_tensors_of_another_device_are_refused(ops, name, wrong):
    f = getattr(ops, name)
    with pytest.raises(FgError) as e:
        f(*made(name, wrong), stream=0)
    assert e.value.status == _lib.FG_EINVAL
    assert not ops.lib.seen


@pytest.mark.parametrize("name", arguments())
def test_tensors_of_the_handles_device_reach_the_library(ops, name):
    getattr(ops, name)(*made(name, None), stream=0)
    assert ops.lib.seen == ["ts_" + name]
