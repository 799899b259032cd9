"""GPU parity of the training-step operators against the oracle in 64 bits, at
the sizes, strides, types and masks where they can go wrong."""
import ctypes as C

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import Checkpoint, FgError, TrainingOps, _lib
from oracle import training as OT

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# Per tensor, max |g - r| / max(|r|, rms(r)).  float32: a row's statistics are
# sums of at most a few dozen terms a thread and a tree across threads, a few
# dozen roundings of 2^-24 in all.  bf16: one rounding to 8 bits of significand,
# 2^-8 at most, on top.
TOL = {F32: 1e-5, BF16: 2.0 ** -8 + 2e-5}


@pytest.fixture(scope="module")
def ops():
    return TrainingOps()


def dev(a, dtype=F32, pad=0):
    """A numpy matrix on the GPU, rows `pad` elements further apart (the gap
    holds NaN: nothing may read it)."""
    a = np.asarray(a)
    buf = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :a.shape[1]] = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()
    return buf[:, :a.shape[1]]


def vec(a):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def empty(shape, dtype=F32, pad=0):
    """An output matrix whose gap must stay as it is."""
    return torch.full((shape[0], shape[1] + pad), -77.0, dtype=dtype, device="cuda")[:, :shape[1]]


def gap_kept(t, pad):
    if pad:
        whole = torch.as_strided(t, (t.shape[0], t.shape[1] + pad), t.stride(), t.storage_offset())
        assert (whole[:, t.shape[1]:] == -77.0).all()


def close(got, ref, tol):
    got, ref = host(got) if isinstance(got, torch.Tensor) else got, np.asarray(ref, np.float64)
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf])
    ok = np.isfinite(ref)
    g, r = got[ok], ref[ok]
    if r.size:
        rms = np.sqrt(np.mean(r * r))
        den = np.maximum(np.abs(r), rms)
        err = np.max(np.abs(g - r) / np.where(den == 0, 1.0, den))
        assert err <= tol, err


def within(got, ref, bound):
    d = np.abs(host(got) - ref)
    assert (d <= bound).all(), (d - bound).max()


def normal(seed, *shape):
    return np.random.default_rng(seed).normal(size=shape).astype(np.float32)


def rounded(a, dtype):
    return host(torch.from_numpy(np.asarray(a, np.float32)).to(dtype))


# ---- layer norm ----------------------------------------------------------------

# one column; ragged warps; each kernel's longest row and one past it; long rows
NORM_SHAPES = [(1, 1), (3, 17), (5, 32), (2, 257), (64, 1024), (7, 1025), (3, 4096), (2, 4104), (2, 5003), (2, 8192),
               (3, 8200), (1, 16384), (2, 16385), (2, 70001)]
TYPES = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]


@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("xt, yt", TYPES)
@pytest.mark.parametrize("rows, cols", NORM_SHAPES)
def test_layer_norm(ops, rows, cols, xt, yt, pad):
    x = rounded(normal(cols, rows, cols) * 1.5 + 0.4, xt)
    gamma, beta = normal(1, cols) * 0.1 + 1, normal(2, cols) * 0.1
    affine = (rows + cols + pad) % 3 != 0
    ref, mean, rstd, h = OT.layer_norm(x, gamma if affine else None, beta if affine else None)
    y = empty((rows, cols), yt, pad)
    m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ck = Checkpoint(rows, cols)
    ck.buf.fill_(0xAA)
    ops.layer_norm(dev(x, xt, pad), vec(gamma) if affine else None, vec(beta) if affine else None, y, m, r, ckpt=ck)
    ops.sync()
    gap_kept(y, pad)
    close(y, ref, TOL[yt])
    close(m, mean, 1e-5)
    close(r, rstd, 1e-5)
    # the saved rows: normalised blocks, each value half a step off at most,
    # the float32 error of h aside; past the last column zeros
    b = ck.buf.cpu().numpy()
    v, step = OT.checkpoint_decode(b, rows, cols), OT.checkpoint_steps(b, rows, cols)
    err = np.abs(v - h)
    assert (err <= np.where(np.abs(h) > 127 * step, step, step / 2) + 2e-5 * np.maximum(1, np.abs(h))).all()
    p = OT.pitch(cols)
    assert not b[:rows * p].reshape(rows, p)[:, cols:].any()
    if cols > 1:
        q = np.abs(b[:rows * p].view(np.int8).astype(int)).reshape(rows, p // 32, 32).max(2)
        assert (q[:, :(cols + 31) // 32] >= 63).all()


@pytest.mark.parametrize("from_ckpt", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("xt, dt", TYPES)
@pytest.mark.parametrize("rows, cols", NORM_SHAPES + [(700, 96), (333, 1001), (1500, 264)])
def test_layer_norm_backward(ops, rows, cols, xt, dt, pad, from_ckpt):
    x = rounded(normal(cols, rows, cols) * 1.5 + 0.4, xt)
    dy = rounded(normal(cols + 1, rows, cols), dt)
    gamma = normal(1, cols) * 0.1 + 1
    affine = (rows + cols + pad) % 3 != 0
    _, mean, rstd, h = OT.layer_norm(x)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    dx = empty((rows, cols), xt, pad)
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    if from_ckpt:
        b = OT.checkpoint_encode(h.astype(np.float32))
        h = OT.checkpoint_decode(b, rows, cols)
        src = Checkpoint(rows, cols, torch.from_numpy(b).cuda())
    else:
        src = dev(x, xt, pad)
        h = (x - mean[:, None].astype(np.float64)) * rstd[:, None]
    g = gamma if affine else None
    ref, rg, rb = OT.layer_norm_backward(dy, h, rstd, g)
    args = (dev(dy, dt, pad), src, None if g is None else vec(g), None if from_ckpt else vec(mean), vec(rstd), dx)
    ops.layer_norm_backward(*args, dg, db)
    ops.sync()
    gap_kept(dx, pad)
    if cols > 1:
        close(dx, ref, TOL[xt])
    else:
        assert np.abs(host(dx)).max() <= 1e-3      # the exact gradient of one column is 0
    # sums over rows: at most rows / 8 + 64 additions one after the other, and
    # h itself is a few roundings off
    n = 2.0 ** -24 * (rows / 8 + 64)
    within(dg, rg, n * np.abs(dy * h).sum(0) + 2.0 ** -22 * (np.abs(dy) * (np.abs(h) + 1)).sum(0) + 1e-30)
    within(db, rb, n * np.abs(dy).sum(0) + 1e-30)
    # the same call again is the same to the bit; accumulated, it doubles
    dx2, dg2, db2 = empty((rows, cols), xt, pad), dg.clone(), db.clone()
    ops.layer_norm_backward(*args[:-1], dx2, dg2, db2, accumulate=True)
    ops.sync()
    assert torch.equal(dx, dx2) and torch.equal(dg2, dg + dg) and torch.equal(db2, db + db)


# long rows, several to an SM
@pytest.mark.parametrize("from_ckpt", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("xt, dt", TYPES)
@pytest.mark.parametrize("rows, cols", [(400, 8200), (170, 16384)])
def test_layer_norm_backward_of_long_rows(ops, rows, cols, xt, dt, pad, from_ckpt):
    test_layer_norm_backward(ops, rows, cols, xt, dt, pad, from_ckpt)


def test_layer_norm_gradient_by_differences(ops):
    # the forward kernel's directional difference against the backward
    # kernel's gradient: float32 outputs differ by 2^-22 or so, over a step of
    # 2^-6 that is 1e-4 of the loss's terms, and the third derivative adds 2e-4
    rows, cols = 5, 300
    x, w, d = normal(1, rows, cols), normal(2, rows, cols), normal(3, rows, cols)
    gamma, beta = vec(normal(4, cols)), vec(normal(5, cols))
    m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

    def loss(v):
        y = empty((rows, cols))
        ops.layer_norm(dev(v), gamma, beta, y, m, r)
        return (host(y) * w).sum()

    h = 2.0 ** -6
    diff = (loss(x + h * d) - loss(x - h * d)) / (2 * h)
    loss(x)
    dx, dg, db = empty((rows, cols)), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ops.layer_norm_backward(dev(w), dev(x), gamma, m, r, dx, dg, db)
    assert abs(diff - (host(dx) * d).sum()) <= 5e-4 * np.abs(host(dx) * d).sum()


def test_layer_norm_of_awkward_rows(ops):
    # constant rows (no variance), a far mean, NaN and infinite values
    x = np.zeros((5, 200), np.float32)
    x[1] = 3.0
    x[2] = 1e4 + normal(0, 200)
    x[3] = normal(1, 200)
    x[3, 7] = np.nan
    x[4] = normal(2, 200)
    x[4, 9] = np.inf
    y, m, r = empty((5, 200)), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    ck = Checkpoint(5, 200)
    ops.layer_norm(dev(x), None, None, y, m, r, ckpt=ck)
    got = host(y)
    assert not got[:2].any()
    ref = OT.layer_norm(x[2:3])[0]
    # the mean of values near 1e4 is known to 1e4 2^-24 times a few roundings
    assert np.abs(got[2] - ref).max() < 1e4 * 2.0 ** -24 * 16
    assert np.isnan(got[3:]).all()
    back = OT.checkpoint_decode(ck.buf.cpu().numpy(), 5, 200)
    assert not back[:2].any() and np.isnan(back[3:, :]).all()


def test_layer_norm_in_place_and_empty(ops):
    x = normal(3, 6, 520)
    t = dev(x)
    ops.layer_norm(t, None, None, t, None, None)
    close(t, OT.layer_norm(x)[0], 1e-5)
    _, mean, rstd, h = OT.layer_norm(x)
    dy = normal(4, 6, 520)
    t = dev(dy)
    ops.layer_norm_backward(t, dev(x), None, vec(mean), vec(rstd), t, None, None)
    close(t, OT.layer_norm_backward(dy, h, rstd)[0], 1e-5)
    none = torch.empty((0, 40), device="cuda")
    z = torch.empty(0, device="cuda")
    ops.layer_norm(none, None, None, none.clone(), z, z)
    dg, db = torch.full((40,), 5.0, device="cuda"), torch.full((40,), 6.0, device="cuda")
    ops.layer_norm_backward(none, none.clone(), None, z, z, none.clone(), dg, db, accumulate=True)
    assert (dg == 5).all() and (db == 6).all()
    ops.layer_norm_backward(none, none.clone(), None, z, z, none.clone(), dg, db)
    assert not dg.any() and not db.any()


# ---- checkpoints ---------------------------------------------------------------

CKPT_SHAPES = [(1, 1), (3, 31), (2, 32), (5, 127), (4, 128), (3, 255), (2, 257), (33, 1000), (2, 4097), (257, 520)]


def awkward(rows, cols):
    """Values of all magnitudes, ties between steps, zeros, subnormals, infinities and NaN."""
    r = np.random.default_rng(cols)
    x = (r.normal(size=(rows, cols)) * np.exp(r.normal(size=(rows, cols)) * 4)).astype(np.float32)
    flat = x.reshape(-1)
    kinds = r.integers(0, 40, size=flat.size)
    flat[kinds == 0] = 0.0
    flat[kinds == 1] = -0.0
    flat[kinds == 2] = 1e-41
    flat[kinds == 3] = 2.5e38
    flat[kinds == 4] = 0.0234375
    if flat.size > 100:
        flat[flat.size // 2] = np.nan
        flat[flat.size // 3] = -np.inf
    return x


@pytest.mark.parametrize("pad", [0, 16, 1])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, cols", CKPT_SHAPES)
def test_checkpoint_bytes(ops, rows, cols, dtype, pad):
    x = rounded(awkward(rows, cols), dtype).astype(np.float32)
    ck = Checkpoint(rows, cols)
    ck.buf.fill_(0xAA)
    ops.checkpoint_save(dev(x, dtype, pad), ck)
    ref = OT.checkpoint_encode(x)
    np.testing.assert_array_equal(ck.buf.cpu().numpy(), ref)
    want = OT.checkpoint_decode(ref, rows, cols)
    for yt in (F32, BF16):          # both hold the values exactly
        y = empty((rows, cols), yt, pad)
        ops.checkpoint_load(ck, y)
        np.testing.assert_array_equal(host(y), want)
        gap_kept(y, pad)


@pytest.mark.parametrize("op", ["relu", "sigmoid", "tanh"])
@pytest.mark.parametrize("dt, xt", TYPES)
@pytest.mark.parametrize("rows, cols, pad", [(1, 1, 0), (3, 31, 0), (5, 257, 1), (33, 1000, 8), (9, 4096, 0)])
def test_activation_backward(ops, op, dt, xt, rows, cols, pad):
    f = {"relu": lambda v: np.maximum(v, 0), "sigmoid": lambda v: 1 / (1 + np.exp(-v)), "tanh": np.tanh}[op]
    a = f(normal(cols, rows, cols))
    if a.size > 64:
        a[0, 3] = np.nan
    b = OT.checkpoint_encode(a)
    dy = rounded(normal(cols + 1, rows, cols), dt)
    dx = empty((rows, cols), xt, pad)
    ops.activation_backward(op, dev(dy, dt, pad), Checkpoint(rows, cols, torch.from_numpy(b).cuda()), dx)
    close(dx, OT.activation_backward(op, dy, OT.checkpoint_decode(b, rows, cols)), TOL[xt])
    gap_kept(dx, pad)


# tokens, columns, outputs: single ones; ragged against every tile; K tails;
# few tiles with many tokens; more tiles than SMs
WGRAD_SHAPES = [(1, 1, 1), (1, 32, 8), (3, 130, 24), (63, 100, 100), (64, 128, 256), (65, 129, 257), (200, 256, 512),
                (130, 384, 136), (1000, 333, 777), (4097, 64, 40), (2048, 256, 256), (96, 2100, 2600), (8192, 160, 264),
                (31, 500, 8), (777, 1024, 1024)]


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 5])
@pytest.mark.parametrize("rows, cols, n", WGRAD_SHAPES)
def test_weight_grad(ops, rows, cols, n, pad, affine):
    b = OT.checkpoint_encode(normal(rows, rows, cols))
    h = OT.checkpoint_decode(b, rows, cols)
    dy = rounded(normal(rows + 1, rows, n) * 0.1, BF16)
    gamma, beta = (normal(1, cols) * 0.1 + 1, normal(2, cols) * 0.1) if affine else (None, None)
    ref, rb = OT.weight_grad(h, dy, gamma, beta)
    dw, db = empty((cols, n), F32, pad), torch.empty(n, device="cuda")
    ck, d = Checkpoint(rows, cols, torch.from_numpy(b).cuda()), dev(dy, BF16, pad)
    more = {} if not affine else {"gamma": vec(gamma), "beta": vec(beta)}
    ops.weight_grad(ck, d, dw, db=db, **more)
    ops.sync()
    gap_kept(dw, pad)
    # products are exact; each addition (whatever the order) is off by 2^-23
    # of its partial sum at most, rows + 8 of them
    size = (np.abs(h) * (1 if gamma is None else np.abs(gamma))).T @ np.abs(dy)
    if beta is not None:
        size += np.abs(beta)[:, None] * np.abs(dy).sum(0)
    within(dw, ref, 2.0 ** -23 * (rows + 8) * size + 1e-30)
    # in the norm the errors average out: the float32 bound of a sum of `rows`
    # terms in random order
    assert np.linalg.norm(host(dw) - ref) <= 2.0 ** -23 * (4 + np.sqrt(rows)) * np.linalg.norm(ref) + 1e-30
    within(db, rb, 2.0 ** -24 * (rows / 8 + 64) * np.abs(dy).sum(0) + 1e-30)
    dw2, db2 = empty((cols, n), F32, pad), db.clone()
    dw2.copy_(dw)
    ops.weight_grad(ck, d, dw2, db=db2, accumulate=True, **more)
    ops.sync()
    gap_kept(dw2, pad)
    assert torch.equal(dw2, dw + dw) and torch.equal(db2, db + db)


# rows of dy off 16 bytes go through a copy in the workspace, here by a few
# hundred and by single tokens at a time; dw in the caller's buffer, with a gap
@pytest.mark.parametrize("rows, cols, n", [(1500, 96, 601), (9, 40, 65535)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_grad_of_unaligned_rows_in_a_small_workspace(rows, cols, n, accumulate):
    ops = TrainingOps(1 << 20)
    b = OT.checkpoint_encode(normal(rows, rows, cols))
    h = OT.checkpoint_decode(b, rows, cols)
    dy = rounded(normal(rows + 1, rows, n) * 0.1, BF16)
    gamma, beta = normal(1, cols) * 0.1 + 1, normal(2, cols) * 0.1
    ref, rb = OT.weight_grad(h, dy, gamma, beta)
    old, oldb = normal(3, cols, n), normal(4, n)
    dw, db = empty((cols, n), F32, 3), vec(oldb)
    dw.copy_(vec(old))
    ops.weight_grad(Checkpoint(rows, cols, torch.from_numpy(b).cuda()), dev(dy, BF16, 2), dw, db=db, gamma=vec(gamma),
                    beta=vec(beta), accumulate=accumulate)
    ops.sync()
    gap_kept(dw, 3)
    base, baseb = (rounded(old, F32), rounded(oldb, F32)) if accumulate else (0.0 * old, 0.0 * oldb)
    # every addition is off by 2^-23 of its partial sum at most: rows + 8, and
    # one to each piece for what is added to
    size = np.abs(h * gamma).T @ np.abs(dy) + np.abs(beta)[:, None] * np.abs(dy).sum(0)
    within(dw, base + ref, 2.0 ** -23 * (2 * rows + 8) * (size + np.abs(base)) + 1e-30)
    within(db, baseb + rb, 2.0 ** -23 * (2 * rows + 64) * (np.abs(dy).sum(0) + np.abs(baseb)) + 1e-30)


def test_weight_grad_of_no_rows_and_marked_blocks(ops):
    dw, db = torch.full((40, 24), 3.0, device="cuda"), torch.full((24,), 3.0, device="cuda")
    ck = Checkpoint(0, 40)
    dy = torch.empty((0, 24), dtype=BF16, device="cuda")
    ops.weight_grad(ck, dy, dw, db=db, beta=torch.ones(40, device="cuda"), accumulate=True)
    ops.sync()
    assert (dw == 3).all() and (db == 3).all()
    ops.weight_grad(ck, dy, dw, db=db)
    ops.sync()
    assert not dw.any() and not db.any()
    # a marked block of a token poisons its 32 rows of dw, nothing else; a NaN
    # in dy its column
    x = normal(5, 70, 100)
    x[40, 50] = np.inf
    dyh = normal(6, 70, 24)
    dyh[3, 5] = np.nan
    b = OT.checkpoint_encode(x)
    dw = torch.empty((100, 24), device="cuda")
    ops.weight_grad(Checkpoint(70, 100, torch.from_numpy(b).cuda()), dev(dyh, BF16), dw)
    bad = np.isnan(host(dw))
    want = np.zeros((100, 24), bool)
    want[32:64] = True
    want[:, 5] = True
    assert np.array_equal(bad, want)


# ---- log probabilities -----------------------------------------------------------


def logits_of(kind, rows, vocab):
    x = normal(vocab, rows, vocab) * 2.5
    if kind == "ties":
        x = np.round(x)
    if kind == "masked":
        x[np.random.default_rng(rows).random((rows, vocab)) < 0.7] = -np.inf
        x[rows // 2] = -np.inf                       # a row of nothing
        x[0] = -np.inf
        x[0, vocab // 2] = -3e38                     # one possible token, the type's lowest value or so
    if kind == "awkward":
        x[0, vocab // 3] = np.nan
        x[rows - 1, vocab // 2] = np.inf
        x[rows // 2] = -0.0
        x[rows // 2, ::3] = 0.0
        x[rows // 3] *= 1000.0
    return x


LOGIT_SHAPES = [(1, 1), (4, 2), (3, 31), (5, 257), (2, 1000), (7, 5003), (300, 128), (3, 32000), (1, 50001), (2, 131072),
                (160, 4097)]


@pytest.mark.parametrize("k", [0, 1, 8, 32])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "awkward"])
@pytest.mark.parametrize("dtype, pad", [(F32, 0), (F32, 3), (BF16, 0), (BF16, 7)])
@pytest.mark.parametrize("rows, vocab", LOGIT_SHAPES)
def test_token_logprobs(ops, rows, vocab, dtype, pad, kind, k):
    if kind == "awkward" and rows < 4:
        pytest.skip("needs four rows")
    x = rounded(logits_of(kind, rows, vocab), dtype)
    k = min(k, vocab)
    tokens = np.random.default_rng(k).integers(-1, vocab + 1, size=rows)
    lp, ent, lse, tlp, ids = OT.token_logprobs(x, tokens, k)
    out = [torch.empty(rows, device="cuda") for _ in range(3)]
    gl = torch.empty((rows, k), device="cuda") if k else None
    gi = torch.empty((rows, k), dtype=torch.int32, device="cuda") if k else None
    ops.token_logprobs(dev(x, dtype, pad), torch.from_numpy(tokens).cuda(), *out, gl, gi)
    for got, ref in zip(out, (lp, ent, lse)):
        # off by a few roundings of the largest logit of the row (its exponent
        # is the difference of two float32 values of that size)
        big = np.where(np.isfinite(x), np.abs(x), 0).max(1)
        g = host(got)
        assert np.array_equal(np.isnan(g), np.isnan(ref)) and np.array_equal(np.isinf(g), np.isinf(ref))
        ok = np.isfinite(ref)
        assert (g[np.isinf(ref)] == ref[np.isinf(ref)]).all()
        assert (np.abs(g[ok] - ref[ok]) <= (2.0 ** -22 * (big + 16) * 4)[ok]).all()
    if k:
        np.testing.assert_array_equal(gi.cpu().numpy(), ids)
        g = host(gl)
        assert np.array_equal(np.isnan(g), np.isnan(tlp)) and np.array_equal(np.isinf(g), np.isinf(tlp))
        ok = np.isfinite(tlp)
        big = np.broadcast_to(np.where(np.isfinite(x), np.abs(x), 0).max(1)[:, None], g.shape)
        assert (np.abs(g[ok] - tlp[ok]) <= (2.0 ** -22 * (big + 16) * 4)[ok]).all()


# more rows than the SMs' blocks at one time: other numbers of warps to a row
@pytest.mark.parametrize("k", [0, 32])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "awkward"])
@pytest.mark.parametrize("dtype, pad", [(F32, 3), (BF16, 7)])
@pytest.mark.parametrize("vocab", [2051, 16384, 16391])
def test_token_logprobs_many_rows(ops, vocab, dtype, pad, kind, k):
    test_token_logprobs(ops, 650, vocab, dtype, pad, kind, k)


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("kind", ["normal", "masked"])
@pytest.mark.parametrize("xt, dt", TYPES)
@pytest.mark.parametrize("rows, vocab, pad", [(1, 1, 0), (4, 2, 0), (5, 257, 1), (7, 5003, 0), (300, 128, 8), (3, 32000, 0)])
def test_token_logprobs_backward(ops, rows, vocab, pad, xt, dt, kind, entropy):
    x = rounded(logits_of(kind, rows, vocab), xt)
    tokens = np.random.default_rng(7).integers(-1, vocab + 1, size=rows)
    g, w = normal(1, rows), normal(2, rows)
    t = torch.from_numpy(tokens).cuda()
    lp, ent, lse = [torch.empty(rows, device="cuda") for _ in range(3)]
    xd = dev(x, xt, pad)
    ops.token_logprobs(xd, t, lp, ent, lse)
    d = empty((rows, vocab), dt, pad)
    ops.token_logprobs_backward(xd, t, lse, ent if entropy else None, vec(g), vec(w) if entropy else None, d)
    ref = OT.token_logprobs_backward(x, tokens, g, w if entropy else None)
    gap_kept(d, pad)
    # p inherits the error of logit - lse: a few roundings of values near 16
    bound = np.abs(ref) * TOL[dt] + 2.0 ** -20 * (np.abs(g) + np.abs(w) * 4)[:, None]
    within(d, ref, bound + 1e-30)
    if xt == dt:
        ops.token_logprobs_backward(xd, t, lse, ent if entropy else None, vec(g), vec(w) if entropy else None, xd)
        assert torch.equal(xd, d)


def test_token_logprobs_gradient_by_differences(ops):
    rows, vocab = 4, 600
    x, d = normal(1, rows, vocab), normal(2, rows, vocab)
    t = torch.tensor([5, 599, 0, -1], device="cuda")
    g, w = normal(3, rows), normal(4, rows)
    lp, ent, lse = [torch.empty(rows, device="cuda") for _ in range(3)]

    def loss(v):
        ops.token_logprobs(dev(v), t, lp, ent, lse)
        return (host(lp) * g).sum() + (host(ent) * w).sum()

    h = 2.0 ** -5
    diff = (loss(x + h * d) - loss(x - h * d)) / (2 * h)
    loss(x)
    dx = empty((rows, vocab))
    ops.token_logprobs_backward(dev(x), t, lse, ent, vec(g), vec(w), dx)
    # values near 6 in float32 over the step, and the third derivative's part
    assert abs(diff - (host(dx) * d).sum()) <= 1e-3 * (np.abs(host(dx) * d).sum() + 1)


# ---- streams, graphs, refusals ----------------------------------------------------


def test_streams_and_graph_replay(ops):
    # inputs made on another stream, the call on a side stream that waits for
    # it; then the same call captured and replayed on new inputs
    rows, cols = 500, 1000
    side = torch.cuda.Stream()
    x, dy = dev(normal(1, rows, cols)), dev(normal(2, rows, cols))
    _, mean, rstd, h = OT.layer_norm(host(x))
    m, r = vec(mean), vec(rstd)
    dx, dg, db = empty((rows, cols)), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    ops.layer_norm_backward(dy, x, None, m, r, dx, dg, db, stream=side)
    ops.sync(side)
    ref = OT.layer_norm_backward(host(dy), h, rstd)
    close(dx, ref[0], 1e-5)
    first = dg.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.layer_norm_backward(dy, x, None, m, r, dx, dg, db)
    dg.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dg, first)
    dy.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dg, first * 2)


def test_two_handles_on_two_streams():
    a, b = TrainingOps(), TrainingOps(1 << 20)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    rows, cols, n = 600, 200, 144
    ck = Checkpoint(rows, cols, torch.from_numpy(OT.checkpoint_encode(normal(1, rows, cols))).cuda())
    dy = dev(normal(2, rows, n), BF16)
    out = [torch.empty((cols, n), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        a.weight_grad(ck, dy, out[0], stream=s)
        b.weight_grad(ck, dy, out[1], stream=t)
    a.sync(s)
    b.sync(t)
    ref = OT.weight_grad(OT.checkpoint_decode(ck.buf.cpu().numpy(), rows, cols), host(dy))[0]
    for o in out:
        assert np.linalg.norm(host(o) - ref) <= 1e-5 * np.linalg.norm(ref)


def refused(status, f, *a, **k):
    with pytest.raises(FgError) as e:
        f(*a, **k)
    assert e.value.status == status, e.value


def test_refusals(ops):
    lib = _lib.load()
    x, y = torch.zeros((4, 64), device="cuda"), torch.zeros((4, 64), device="cuda")
    v, s = torch.zeros(64, device="cuda"), torch.zeros(4, device="cuda")
    ck = Checkpoint(4, 64)
    E, S, U = _lib.FG_EINVAL, _lib.FG_ESHAPE, _lib.FG_EUNSUPPORTED
    refused(E, ops.layer_norm, x.half(), None, None, y, s, s)
    refused(E, ops.layer_norm, x.cpu(), None, None, y, s, s)
    refused(S, ops.layer_norm, x, None, None, y[:, :32], s, s)
    refused(S, ops.layer_norm, x, v[:32], None, y, s, s)
    refused(E, ops.layer_norm, x, v.double(), None, y, s, s)
    refused(E, ops.layer_norm, x.t().contiguous().t(), None, None, y, s, s)
    refused(E, ops.layer_norm, x, None, None, y, s, s, eps=-1.0)
    refused(E, ops.layer_norm, x, None, None, y, s, s, eps=float("nan"))
    refused(S, ops.layer_norm, x, None, None, y, s, s, ckpt=Checkpoint(4, 65))
    refused(E, ops.layer_norm_backward, x, x, None, None, s, y, v, v)
    refused(E, ops.layer_norm_backward, x, x, None, s, s, y.bfloat16(), v, v)
    refused(E, ops.layer_norm_backward, x, ck, None, None, None, y, v, v)
    refused(S, ops.checkpoint_save, x[:3], ck)
    refused(E, Checkpoint, 4, 64, torch.zeros(10, dtype=torch.uint8, device="cuda"))
    refused(S, Checkpoint, 4, 0)
    refused(E, ops.activation_backward, "exp", x, ck, y)
    refused(E, ops.weight_grad, ck, x, torch.zeros((64, 64), device="cuda"))
    refused(E, ops.weight_grad, ck, x.bfloat16(), torch.zeros((64, 64), dtype=BF16, device="cuda"))
    refused(S, ops.weight_grad, ck, x.bfloat16(), torch.zeros((64, 63), device="cuda"))
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    refused(E, ops.token_logprobs, x, t.int(), s, s, s)
    refused(E, ops.token_logprobs, x, None, s, s, s)
    refused(E, ops.token_logprobs, x, t, s, s, s, torch.zeros((4, 33), device="cuda"),
            torch.zeros((4, 33), dtype=torch.int32, device="cuda"))
    refused(E, ops.token_logprobs, x[:, :3], t, s, s, s, torch.zeros((4, 4), device="cuda"),
            torch.zeros((4, 4), dtype=torch.int32, device="cuda"))
    refused(E, ops.token_logprobs, x, t, s, s, s, torch.zeros((4, 2), device="cuda"))
    refused(E, ops.token_logprobs_backward, x, t, None, None, s, None, y)
    refused(E, ops.token_logprobs_backward, x, t, s, None, s, s, y)
    refused(E, TrainingOps, -1)
    refused(E, TrainingOps, 1000)
    wide = torch.zeros((1, 100_000), device="cuda")
    small, sv = TrainingOps(1 << 20), torch.zeros(1, device="cuda")
    refused(U, small.layer_norm_backward, wide, wide, None, sv, sv, wide.clone(), None, None)
    # below the binding: misaligned pointers, short pitches, unknown types
    p, h = C.c_void_p(x.data_ptr()), ops.h
    assert lib.ts_layer_norm(h, C.c_void_p(x.data_ptr() + 2), 0, 64, 4, 64, None, None, 1e-5, y.data_ptr(), 0, 64, None,
                             None, None, None) == E
    assert lib.ts_layer_norm(h, p, 0, 63, 4, 64, None, None, 1e-5, y.data_ptr(), 0, 64, None, None, None, None) == S
    assert lib.ts_layer_norm(h, p, 7, 64, 4, 64, None, None, 1e-5, y.data_ptr(), 0, 64, None, None, None, None) == E
    assert lib.ts_layer_norm(h, None, 0, 64, 4, 64, None, None, 1e-5, y.data_ptr(), 0, 64, None, None, None, None) == E
    assert lib.ts_checkpoint_save(h, p, 0, 64, 4, 64, C.c_void_p(ck.ptr + 8), None) == E
    assert lib.ts_weight_grad(h, ck.ptr, 4, 64, None, None, p, 1, 64, 1 << 21, p, 1 << 21, None, 0, None) in (S, U)
    ops.sync()


# ---- the operators together --------------------------------------------------------


def test_training_step_example():
    from examples import training_step as T
    m = T.Model(tokens=200, width=96, hidden=160, vocab=328, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((200, 96), generator=gen, device="cuda")
    t = torch.randint(0, 328, (200,), generator=gen, device="cuda")
    loss = m.step(x, t)
    m.ops.sync()
    # the same step in 64 bits, rounded where the step rounds: the matmuls'
    # operands to bf16, the saved activations to 8 bits
    gamma, beta, w1, b1, w2 = (host(p) for p in m.params)
    w1, w2 = rounded(w1, BF16), rounded(w2, BF16)
    y, _, rstd, h = OT.layer_norm(host(x), gamma, beta)
    saved_norm = OT.checkpoint_decode(OT.checkpoint_encode(h), 200, 96)
    acts = np.maximum(rounded(y, BF16) @ w1 + b1, 0)
    saved_acts = OT.checkpoint_decode(OT.checkpoint_encode(acts), 200, 160)
    logits, tokens = saved_acts @ w2, t.cpu().numpy()
    want_loss = -OT.token_logprobs(logits, tokens)[0].mean()
    dlogits = rounded(OT.token_logprobs_backward(logits, tokens, np.full(200, -1.0 / 200)), BF16)
    dw2 = OT.weight_grad(saved_acts, dlogits)[0]
    dhidden = rounded(OT.activation_backward("relu", dlogits @ w2.T, saved_acts), BF16)
    dw1, db1 = OT.weight_grad(saved_norm, dhidden, gamma, beta)
    dx, dgamma, dbeta = OT.layer_norm_backward(dhidden @ w1.T, saved_norm, rstd, gamma)
    assert abs(loss.item() - want_loss) < 1e-4 * want_loss
    # a value that lies on the edge of its rounding may go the other way, 2^-8
    # of itself in bf16: were it all of them, that is what the results are off
    for got, want in zip(m.grads + [m.dx], [dgamma, dbeta, dw1, db1, dw2, dx]):
        assert np.linalg.norm(host(got) - want) <= 2.0 ** -8 * np.linalg.norm(want)


def test_training_example_learns():
    from examples import training_step as T
    losses = T.main(steps=12)
    assert losses[-1] < 0.9 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
