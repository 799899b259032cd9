"""GPU parity of the training-step operators where their loops, aliases and
rounding can go wrong: outputs in place of inputs, rows of every kernel that
walks several, confident rows of logits, empty checkpoints, expired waits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import Checkpoint
from oracle import training as OT
from tests.test_gpu_training import BF16, F32, TOL, close, dev, empty, gap_kept, host, normal, ops, rounded, vec, within  # noqa: F401

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
