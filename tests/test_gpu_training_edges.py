"""GPU parity of the training-step operators where their loops, aliases and
rounding can go wrong: outputs in place of inputs, rows of every kernel that
walks several, confident rows of logits, empty checkpoints, expired waits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import Checkpoint, _lib
from oracle import training as OT
from tests.test_gpu_training import BF16, F32, TOL, close, dev, empty, gap_kept, host, normal, ops, refused, rounded, vec, within  # noqa: F401, E501

pytestmark = pytest.mark.gpu


# ---- in place ------------------------------------------------------------------


# a length of each kernel: one pass, G = 2, the column sums in shared memory,
# the two kernels of longer rows
@pytest.mark.parametrize("from_ckpt", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("rows, cols", [(5, 520), (3, 5003), (3, 8200), (2, 16385), (300, 17000), (2, 70001)])
def test_layer_norm_backward_in_place(ops, rows, cols, pad, dtype, from_ckpt):  # noqa: F811
    x = rounded(normal(cols, rows, cols) * 1.5 + 0.4, dtype)
    dy = rounded(normal(cols + 1, rows, cols), dtype)
    gamma = normal(1, cols) * 0.1 + 1
    _, mean, rstd, h = OT.layer_norm(x)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    if from_ckpt:
        b = OT.checkpoint_encode(h.astype(np.float32))
        h = OT.checkpoint_decode(b, rows, cols)
        src = Checkpoint(rows, cols, torch.from_numpy(b).cuda())
    else:
        src = dev(x, dtype, pad)
        h = (x - mean[:, None].astype(np.float64)) * rstd[:, None]
    ref, rg, rb = OT.layer_norm_backward(dy, h, rstd, gamma)
    t = empty((rows, cols), dtype, pad)
    t.copy_(dev(dy, dtype))
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ops.layer_norm_backward(t, src, vec(gamma), None if from_ckpt else vec(mean), vec(rstd), t, dg, db)
    ops.sync()
    gap_kept(t, pad)
    close(t, ref, TOL[dtype])
    # as where dx is a matrix of its own: at most rows / 8 + 64 additions one
    # after the other, and h is a few roundings off
    n = 2.0 ** -24 * (rows / 8 + 64)
    within(dg, rg, n * np.abs(dy * h).sum(0) + 2.0 ** -22 * (np.abs(dy) * (np.abs(h) + 1)).sum(0) + 1e-30)
    within(db, rb, n * np.abs(dy).sum(0) + 1e-30)


@pytest.mark.parametrize("op", ["relu", "sigmoid", "tanh"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, cols, pad", [(1, 1, 0), (5, 257, 1), (700, 1000, 8), (300, 4096, 0)])
def test_activation_backward_in_place(ops, op, dtype, rows, cols, pad):  # noqa: F811
    a = {"relu": lambda v: np.maximum(v, 0), "sigmoid": lambda v: 1 / (1 + np.exp(-v)), "tanh": np.tanh}[op](normal(cols, rows, cols))
    b = OT.checkpoint_encode(a)
    dy = rounded(normal(cols + 1, rows, cols), dtype)
    t = empty((rows, cols), dtype, pad)
    t.copy_(dev(dy, dtype))
    ops.activation_backward(op, t, Checkpoint(rows, cols, torch.from_numpy(b).cuda()), t)
    close(t, OT.activation_backward(op, dy, OT.checkpoint_decode(b, rows, cols)), TOL[dtype])
    gap_kept(t, pad)


def test_in_place_needs_the_same_type_and_pitch(ops):  # noqa: F811
    # one buffer of 64 rows' room, seen as float32 and bf16 and at two pitches
    x = torch.zeros((64, 64), device="cuda")
    as_bf16, narrow = x.view(BF16)[:32, :32], x[:32, :32]
    wide = torch.as_strided(x, (32, 32), (128, 1))
    s = torch.zeros(32, device="cuda")
    ck, E = Checkpoint(32, 32, torch.zeros(32 * 132, dtype=torch.uint8, device="cuda")), _lib.FG_EINVAL
    for y in (as_bf16, wide):
        refused(E, ops.layer_norm, narrow, None, None, y, s, s)
        refused(E, ops.layer_norm_backward, y, ck, None, None, s, narrow, None, None)
        refused(E, ops.activation_backward, "tanh", narrow, ck, y)
        refused(E, ops.token_logprobs_backward, narrow, torch.zeros(32, dtype=torch.int64, device="cuda"), s, None, s, None, y)
    # a single row has no pitch; the same rows are fine
    ops.layer_norm(narrow[:1], None, None, wide[:1], None, None)
    ops.activation_backward("tanh", narrow, ck, narrow)
    ops.sync()
