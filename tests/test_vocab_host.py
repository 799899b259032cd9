"""The vocabulary operators' checks on the host: tensors of another device, wrong
types and shapes never reach the library; the workspace query."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import FgError, TrainingOps, _lib, linear_cross_entropy_workspace
from tests.test_training_host import Calls, OnDevice


@pytest.fixture
def ops():
    o = TrainingOps.__new__(TrainingOps)
    o.lib, o.h, o.device = Calls(), None, 0
    return o


def arguments():
    """Every call with its tensors: 4 tokens, 64 columns, 9 in the vocabulary."""
    def rows(d=0): return OnDevice((4, 64), torch.bfloat16, d)
    def table(d=0): return OnDevice((9, 64), torch.bfloat16, d)
    def ids(d=0): return OnDevice((4,), torch.int64, d)
    def row(d=0): return OnDevice((4,), device=d)
    return {
        "embedding": (ids, table, rows),
        "embedding_backward": (ids, rows, table),
        "linear_cross_entropy": (rows, table, ids, row, row),
        "linear_cross_entropy_backward": (rows, table, ids, row, row, rows, table, row),
    }


# the arguments that say how large the vocabulary is
TABLES = [("embedding", 1), ("embedding_backward", 2), ("linear_cross_entropy", 1)]
CASES = [(name, i) for name, args in arguments().items() for i in range(len(args))]


@pytest.mark.parametrize("name, wrong", CASES)
def test_tensors_of_another_device_are_refused(ops, name, wrong):
    args = [a(int(i == wrong)) for i, a in enumerate(arguments()[name])]
    with pytest.raises(FgError) as e:
        getattr(ops, name)(*args, stream=0)
    assert e.value.status == _lib.FG_EINVAL and ops.lib.seen == []


@pytest.mark.parametrize("name, wrong", CASES)
def test_wrong_types_and_shapes_are_refused(ops, name, wrong):
    good = arguments()[name]
    t = good[wrong]().t
    for other in (OnDevice(t.shape, torch.float16), OnDevice((*t.shape, 1), t.dtype),
                  OnDevice((t.shape[0] + 1, *t.shape[1:]), t.dtype)):
        args = [a() for a in good]
        args[wrong] = other
        if (name, wrong) in TABLES and other.shape[1:] == t.shape[1:] and other.dtype == t.dtype:
            continue   # (another vocabulary is no error)
        with pytest.raises((FgError, ValueError)) as e:
            getattr(ops, name)(*args, stream=0)
        assert ops.lib.seen == [], e.value


def test_calls_reach_the_library(ops):
    for name, args in arguments().items():
        getattr(ops, name)(*[a() for a in args], stream=0)
    assert ops.lib.seen == ["ts_" + n for n in arguments()]
    a = [f() for f in arguments()["linear_cross_entropy_backward"]]
    ops.linear_cross_entropy_backward(*a[:5], None, None, stream=0)
    ops.linear_cross_entropy(a[0], a[1], None, None, a[3], stream=0)


def test_workspace():
    for rows, cols, vocab in ((1, 1, 1), (16, 1024, 32000), (8192, 4096, 50001), (1 << 20, 64, 1 << 20)):
        least, most = linear_cross_entropy_workspace(rows, cols, vocab)
        # at least the sums of dx, its copy of x and d for 256 of the vocabulary
        assert rows * cols * 6 + rows * 512 <= least <= most
        assert most >= rows * vocab * 2
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0)):
        with pytest.raises(FgError) as e:
            linear_cross_entropy_workspace(*bad)
        assert e.value.status == _lib.FG_ESHAPE
    with pytest.raises(FgError) as e:
        linear_cross_entropy_workspace((1 << 20) + 1, 1, 1)
    assert e.value.status == _lib.FG_EUNSUPPORTED


def test_entry_points_refuse_a_null_handle(lib):
    p, i, f = C.c_void_p(256), 4, 1.0
    for call in (lambda: lib.ts_embedding(None, p, i, p, 0, i, i, i, f, p, 0, i, None),
                 lambda: lib.ts_embedding_backward(None, p, p, 0, i, i, i, i, f, p, 0, i, 0, None),
                 lambda: lib.ts_linear_cross_entropy(None, p, i, p, i, 1, i, i, i, p, p, p, None),
                 lambda: lib.ts_linear_cross_entropy_backward(None, p, i, p, i, 1, i, i, i, p, p, p, p, p, 1, i, p, 1, i, 0,
                                                              None)):
        assert call() == _lib.FG_EINVAL and b"null handle" in lib.fg_last_error()
