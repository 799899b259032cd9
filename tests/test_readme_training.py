"""README's step of a training loop runs as it is printed."""
import os
import textwrap

import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import linear_cross_entropy_workspace

ROWS, WIDTH, VOCAB = 8192, 4096, 50001


def printed():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    text = open(path).read().split("The operators of a training step work on tensors directly:\n")[1]
    lines = text.split("\n")[1:]
    end = next(i for i, s in enumerate(lines) if s and not s.startswith("    "))
    return textwrap.dedent("\n".join(lines[:end]))


def test_the_workspace_is_large_enough():
    """The handle is made with what the sequence's gradient needs (host only)."""
    code = printed()
    made = {}

    def ops(workspace_bytes=0):
        made["bytes"] = workspace_bytes or 64 << 20
    lines = code.split("\n")
    stop = next(i for i, s in enumerate(lines) if "= TrainingOps(" in s)
    names = {"vocab": VOCAB}
    exec(lines[0], names)
    names["TrainingOps"] = ops
    exec("\n".join(lines[1:stop + 1]), names)
    assert made["bytes"] >= linear_cross_entropy_workspace(ROWS, WIDTH, VOCAB)[0]


@pytest.mark.gpu
def test_the_sequence_runs():
    f32, bf16 = dict(device="cuda"), dict(device="cuda", dtype=torch.bfloat16)
    ids, targets = torch.randint(0, VOCAB, (2, ROWS), device="cuda")
    names = dict(
        vocab=VOCAB, width=WIDTH, x=torch.randn((ROWS, WIDTH), device="cuda").to(torch.bfloat16),
        gamma=torch.ones(WIDTH, **f32), beta=torch.zeros(WIDTH, **f32), y=torch.empty((ROWS, WIDTH), **bf16),
        mean=torch.empty(ROWS, **f32), rstd=torch.empty(ROWS, **f32),
        dy=torch.randn((ROWS, WIDTH), device="cuda").to(torch.bfloat16),
        dw=torch.empty((WIDTH, WIDTH), **f32), db=torch.empty(WIDTH, **f32), logits=torch.randn((ROWS, VOCAB), **f32),
        tokens=ids, logprob=torch.empty(ROWS, **f32), entropy=torch.empty(ROWS, **f32), lse=torch.empty(ROWS, **f32),
        top_logprob=torch.empty((ROWS, 20), **f32), top_id=torch.empty((ROWS, 20), device="cuda", dtype=torch.int32),
        ids=ids, table=(torch.randn((VOCAB, WIDTH), device="cuda") / WIDTH ** 0.5).to(torch.bfloat16), targets=targets,
        loss=torch.empty(ROWS, **f32), g_loss=torch.full((ROWS,), 1.0 / ROWS, **f32),
        dx=torch.empty((ROWS, WIDTH), **bf16),
        dtable=torch.empty((VOCAB, WIDTH), **f32))
    exec(printed(), names)
    for out in ("y", "dw", "db", "logprob", "loss", "dx", "dtable"):
        assert names[out].isfinite().all()
    assert names["dtable"].any() and names["dw"].any()
