"""The oracle of the vocabulary operators: its gradients against differences,
and hand-made values."""
import numpy as np

from oracle import training as OT


def test_embedding_of_padded_places():
    table = np.arange(12.0).reshape(4, 3)
    y = OT.embedding([2, -1, 0, 4, 2], table, 0.5)
    assert np.array_equal(y, [[3, 3.5, 4], [0, 0, 0], [0, 0.5, 1], [0, 0, 0], [3, 3.5, 4]])
    d = OT.embedding_backward([2, -1, 0, 4, 2], np.ones((5, 3)) * [[1], [2], [4], [8], [16]], 4, 0.5)
    assert np.array_equal(d, np.ones((4, 3)) * [[2], [0], [8.5], [0]])


def test_embedding_gradient_is_the_differences():
    rng = np.random.default_rng(0)
    ids, table, dy = [3, 1, 3, -1, 0], rng.normal(size=(5, 4)), rng.normal(size=(5, 4))
    d = OT.embedding_backward(ids, dy, 5, 1.5)
    for v in range(5):
        for c in range(4):
            e = np.zeros_like(table)
            e[v, c] = 1e-3
            up, down = ((OT.embedding(ids, table + s * e, 1.5) * dy).sum() for s in (1, -1))
            assert abs((up - down) / 2e-3 - d[v, c]) < 1e-9


def test_loss_of_equal_logits():
    loss, lse = OT.linear_cross_entropy(np.zeros((3, 2)), np.ones((8, 2)), [0, 7, 8])
    assert np.allclose(loss, [np.log(8), np.log(8), 0]) and np.allclose(lse, np.log(8))


def test_loss_gradient_is_the_differences():
    rng = np.random.default_rng(1)
    x, w, targets = rng.normal(size=(5, 4)), rng.normal(size=(7, 4)), [3, -1, 0, 7, 3]
    g, h = rng.normal(size=5), rng.normal(size=5)

    def total(x, w, h):
        loss, lse = OT.linear_cross_entropy(x, w, targets)
        return (loss * g).sum() + (0 if h is None else (lse * h).sum())

    for hh in (None, h):
        _, lse = OT.linear_cross_entropy(x, w, targets)
        dx, dw, d = OT.linear_cross_entropy_backward(x, w, targets, lse, g, hh)
        assert hh is not None or not d[[1, 3]].any()
        for a, da in ((x, dx), (w, dw)):
            for i in np.ndindex(a.shape):
                e = np.zeros_like(a)
                e[i] = 1e-5
                up, down = (total(x + s * e, w, hh) if a is x else total(x, w + s * e, hh) for s in (1, -1))
                assert abs((up - down) / 2e-5 - da[i]) < 1e-8
