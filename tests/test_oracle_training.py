"""Pins of the training-step oracle: gradients against central differences in
float64, the 8-bit encoding against hand-worked blocks, log probabilities
against closed forms; and the host side of the library's checkpoint layout."""
import numpy as np
import pytest

from oracle import training as OT
from group_execution_gb300 import FgError, _lib, checkpoint_layout


def _differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_layer_norm_gradient_by_differences():
    r = np.random.default_rng(0)
    x, w = r.normal(size=(3, 7)), r.normal(size=(3, 7))
    gamma, beta = r.normal(size=7), r.normal(size=7)
    _, _, rstd, h = OT.layer_norm(x, gamma, beta)
    dx, dg, db = OT.layer_norm_backward(w, h, rstd, gamma)
    # central differences of step h are off by about h^2 = 1e-10 and
    # eps / h = 2e-11 of the loss's size
    assert np.abs(dx - _differences(lambda v: (OT.layer_norm(v, gamma, beta)[0] * w).sum(), x)).max() < 1e-8
    assert np.abs(dg - _differences(lambda v: (OT.layer_norm(x, v, beta)[0] * w).sum(), gamma)).max() < 1e-8
    assert np.abs(db - _differences(lambda v: (OT.layer_norm(x, gamma, v)[0] * w).sum(), beta)).max() < 1e-8


def test_logprob_gradient_by_differences():
    r = np.random.default_rng(1)
    x = r.normal(size=(3, 6)) * 2
    tokens, g, w = [4, 0, -1], r.normal(size=3), r.normal(size=3)

    def loss(v):
        lp, ent = OT.token_logprobs(v, tokens)[:2]
        return (lp * g).sum() + (ent * w).sum()

    assert np.abs(OT.token_logprobs_backward(x, tokens, g, w) - _differences(loss, x)).max() < 1e-8


@pytest.mark.parametrize("op", ["sigmoid", "tanh"])
def test_activation_gradient_by_differences(op):
    f = {"sigmoid": lambda v: 1 / (1 + np.exp(-v)), "tanh": np.tanh}[op]
    x, dy = np.linspace(-3, 3, 11)[None], np.linspace(1, 2, 11)[None]
    want = _differences(lambda v: (f(v) * dy).sum(), x)
    assert np.abs(OT.activation_backward(op, dy, f(x)) - want).max() < 1e-8


def test_weight_grad_is_the_affine_product():
    r = np.random.default_rng(2)
    h, dy, g, b = r.normal(size=(5, 4)), r.normal(size=(5, 3)), r.normal(size=4), r.normal(size=4)
    dw, db = OT.weight_grad(h, dy, g, b)
    assert np.allclose(dw, g[:, None] * (h.T @ dy) + b[:, None] * db, rtol=1e-12)


def test_checkpoint_of_worked_blocks():
    x = np.zeros((1, 160), np.float32)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 1.0, -1.984375, 0.0078125, 0.0234375   # step 2^-6: 64, -127, 0.5, 1.5
    x[0, 32], x[0, 33] = 1.999, 0.5                                             # rounds past 127: clamped
    x[0, 64], x[0, 65] = np.inf, 3.0
    x[0, 96] = 1e-42
    x[0, 128] = 3.0e38
    b = OT.checkpoint_encode(x)
    q, e = b[:256].view(np.int8), b[256:]
    assert list(q[:4]) == [64, -127, 0, 2] and e[0] == 127
    assert list(q[32:34]) == [127, 32] and e[1] == 127
    assert e[2] == 255 and not q[64:96].any()
    assert e[3] == 7 and q[96] == 0
    assert e[4] == 254 and q[128] == round(3.0e38 / 2.0 ** 121)
    v = OT.checkpoint_decode(b, 1, 160)
    assert v[0, 1] == -1.984375 and np.isnan(v[0, 64:96]).all() and v[0, 130] == 0


def test_checkpoint_error_is_half_a_step_at_most():
    r = np.random.default_rng(3)
    x = (r.normal(size=(9, 100)) * np.exp(r.normal(size=(9, 100)) * 3)).astype(np.float32)
    b = OT.checkpoint_encode(x)
    v, step = OT.checkpoint_decode(b, 9, 100), OT.checkpoint_steps(b, 9, 100)
    # half a step of rounding; a value above 127 steps (below 128) is clamped
    assert (np.abs(v - x) <= np.where(np.abs(x) > 127 * step, step, step / 2)).all()
    top = np.abs(x).reshape(9, -1)[:, :96].reshape(9, 3, 32).max(2)
    assert (top / step[:, :96:32] >= 64).all() and (top / step[:, :96:32] < 128).all()
    assert np.array_equal(v, v.astype(np.float32))


def test_logprobs_closed_forms():
    x = np.full((4, 8), -np.inf)
    x[0] = 0.0                       # uniform
    x[1, 2] = 5.0                    # one possible token
    x[3, [1, 6]] = 3.0               # two equal tokens
    lp, ent, lse, tlp, ids = OT.token_logprobs(x, [3, 2, 0, 9], 3)
    assert np.allclose(lp, [-np.log(8), 0, -np.inf, 0]) and np.allclose(ent, [np.log(8), 0, 0, np.log(2)])
    assert lse[2] == -np.inf and list(ids[0]) == [0, 1, 2] and list(ids[2]) == [0, 1, 2] and list(ids[3]) == [1, 6, 0]
    assert np.allclose(tlp[3], [-np.log(2), -np.log(2), -np.inf])
    assert not OT.token_logprobs_backward(x, [3, 2, 0, 9], np.ones(4), np.ones(4))[2].any()


@pytest.mark.parametrize("rows, cols", [(0, 1), (1, 1), (3, 127), (2, 128), (5, 129), (7, 4096)])
def test_checkpoint_layout(rows, cols):
    p = OT.pitch(cols)
    assert checkpoint_layout(rows, cols) == (p, rows * p, rows * p + rows * p // 32)
    if rows:
        assert OT.checkpoint_encode(np.ones((rows, cols), np.float32)).size == rows * p // 32 * 33


def test_layout_and_handle_refusals():
    for rows, cols in [(-1, 4), (4, 0), (4, 1 << 31)]:
        with pytest.raises(FgError) as e:
            checkpoint_layout(rows, cols)
        assert e.value.status == _lib.FG_ESHAPE
    lib = _lib.load()
    assert lib.ts_create(0, None) == _lib.FG_EINVAL
    assert lib.ts_sync_status(None, None) == _lib.FG_EINVAL
    assert lib.ts_checkpoint_save(None, None, 0, 4, 1, 4, None, None) == _lib.FG_EINVAL
    lib.ts_destroy(None)
