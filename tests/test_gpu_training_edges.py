"""GPU parity of the training-step operators where their loops, aliases and
rounding can go wrong: outputs in place of inputs, rows of every kernel that
walks several, confident rows of logits, empty checkpoints, expired waits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import Checkpoint, TrainingOps, _lib
from oracle import training as OT
from tests.test_gpu_training import (BF16, F32, TOL, close, dev, empty, gap_kept, host, normal, ops,  # noqa: F401
                                     refused, rounded, vec, within)

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
    f = {"relu": lambda v: np.maximum(v, 0), "sigmoid": lambda v: 1 / (1 + np.exp(-v)), "tanh": np.tanh}[op]
    a = f(normal(cols, rows, cols))
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
    s, t = torch.zeros(32, device="cuda"), torch.zeros(32, dtype=torch.int64, device="cuda")
    ck, E = Checkpoint(32, 32, torch.zeros(32 * 132, dtype=torch.uint8, device="cuda")), _lib.FG_EINVAL
    for y in (as_bf16, wide):
        refused(E, ops.layer_norm, narrow, None, None, y, s, s)
        refused(E, ops.layer_norm_backward, y, ck, None, None, s, narrow, None, None)
        refused(E, ops.activation_backward, "tanh", narrow, ck, y)
        refused(E, ops.token_logprobs_backward, narrow, t, s, None, s, None, y)
    # a single row has no pitch; the same rows are fine
    ops.layer_norm(narrow[:1], None, None, wide[:1], None, None)
    ops.activation_backward("tanh", narrow, ck, narrow)
    ops.sync()


# ---- log probabilities ------------------------------------------------------------


def peaked(kind, rows, vocab):
    """Confident rows: one logit in the row's last tenth lies 0.5 to 31 above
    the rest; or all logits in rising order."""
    r = np.random.default_rng(vocab + rows)
    x = (r.normal(size=(rows, vocab)) * 2.5).astype(np.float32)
    if kind == "rising":
        return np.sort(x * r.uniform(0.1, 12, size=(rows, 1)).astype(np.float32), axis=1)
    at = r.integers(vocab - vocab // 10 - 1, vocab, size=rows)
    x[np.arange(rows), at] = x.max(1) + r.uniform(0.5, 31, size=rows)
    return x


# a row cut over a cluster, eight warps, four warps, one warp to a row
@pytest.mark.parametrize("k", [0, 20])
@pytest.mark.parametrize("kind", ["late", "rising"])
@pytest.mark.parametrize("dtype, pad", [(F32, 0), (F32, 3), (BF16, 7)])
@pytest.mark.parametrize("rows, vocab", [(64, 50001), (650, 16391), (650, 5003), (2500, 1500)])
def test_token_logprobs_of_confident_rows(ops, rows, vocab, dtype, pad, kind, k):  # noqa: F811
    x = rounded(peaked(kind, rows, vocab), dtype)
    tokens = x.argmax(1)
    tokens[::3] = np.random.default_rng(1).integers(0, vocab, size=len(tokens[::3]))
    lp, ent, lse, tlp, ids = OT.token_logprobs(x, tokens, k)
    out = [torch.empty(rows, device="cuda") for _ in range(3)]
    gl = torch.empty((rows, k), device="cuda") if k else None
    gi = torch.empty((rows, k), dtype=torch.int32, device="cuda") if k else None
    ops.token_logprobs(dev(x, dtype, pad), torch.from_numpy(tokens).cuda(), *out, gl, gi)
    glp, gent, glse = (host(o) for o in out)
    # With the sums about a reference within 1 of the row's largest logit, s =
    # sum e^(x - m) is at most a few times its largest term: a thread adds 4
    # values a chunk (at most 16 chunks here), then come at most 24 joins, each
    # addition 2^-24 of s off.  ln s and t / s are then about 1 + H, a dozen
    # roundings of 2^-24.  An exponential's own error (2^-22, and 2^-23 of its
    # argument, at most 64 where it counts) enters the entropy times p |log p|.
    unit = 2.0 ** -24 * (4 * 16 + 24 + 12 + (4 + 128) * ent)
    assert (np.abs(gent - ent) <= unit).all(), np.max((np.abs(gent - ent) / unit))
    assert (gent >= 0).all()
    # lse = m + ln s, and x - lse: two roundings of numbers of that size more
    big = np.abs(x).max(1)
    assert (np.abs(glse - lse) <= unit + 2.0 ** -23 * (big + 16)).all()
    assert (np.abs(glp - lp) <= unit + 2.0 ** -22 * (big + 16)).all()
    if k:
        np.testing.assert_array_equal(gi.cpu().numpy(), ids)
        assert (np.abs(host(gl) - tlp) <= (unit + 2.0 ** -22 * (big + 16))[:, None]).all()


@pytest.mark.parametrize("k", [1, 32])
@pytest.mark.parametrize("rows, vocab", [(1, 1 << 27), (3, 400_003), (700, 40_000)])
def test_top_logits_of_rising_rows(ops, rows, vocab, k):  # noqa: F811
    # Every chunk lies above those before it, so none can be left out by them:
    # a row is read again until a bound from a sample leaves few enough, about
    # four times at most here.  An atomic for each noted chunk makes a reading
    # a few times longer than one of random logits.
    rising = (torch.arange(vocab, device="cuda") * (30.0 / vocab)).expand(rows, vocab).contiguous()
    random = torch.randn((rows, vocab), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ids, lp = torch.empty((rows, k), dtype=torch.int32, device="cuda"), torch.empty((rows, k), device="cuda")

    def microseconds(x):
        times = []
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            ops.token_logprobs(x, None, None, None, None, lp, ids)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return sorted(times)[1]

    fast, slow = microseconds(random), microseconds(rising)
    # equal logits (float32 has fewer values than the row): lowest column first
    want = torch.sort(rising[0], descending=True, stable=True)[1][:k].to(torch.int32)
    assert torch.equal(ids, want.expand(rows, k))
    assert slow <= 50 * fast, (slow, fast)


# ---- no rows --------------------------------------------------------------------


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [40, 17000])
def test_layer_norm_backward_from_an_empty_checkpoint(ops, cols, dtype, accumulate):  # noqa: F811
    dy, s = torch.empty((0, cols), dtype=dtype, device="cuda"), vec([])
    dx = dy.clone()
    dg, db = torch.full((cols,), 5.0, device="cuda"), torch.full((cols,), 6.0, device="cuda")
    ops.layer_norm_backward(dy, Checkpoint(0, cols), None, None, s, dx, dg, db, accumulate=accumulate)
    ops.sync()
    assert (dg == (5 if accumulate else 0)).all() and (db == (6 if accumulate else 0)).all()


# ---- expired waits ---------------------------------------------------------------


# one tile; pieces of tiles; whole tiles of two accumulations; rows of dy that
# go through a copy
@pytest.mark.parametrize("rows, cols, n, pad", [(300, 200, 144, 0), (3000, 600, 700, 8), (2300, 2560, 2304, 0),
                                                (1000, 333, 777, 5)])
def test_weight_grad_reports_an_expired_wait(rows, cols, n, pad):
    # no copy is ever issued, so every wait runs out after 1 ms: the kernel
    # gives its tensor memory back and returns, the handle reports it once, and
    # the next calls of this and of another handle are right
    stuck = TrainingOps(wait_limit_ns=1_000_000, flags=_lib.FG_FLAG_INJECT_NO_LOADS)
    b = OT.checkpoint_encode(normal(rows, rows, cols))
    h = OT.checkpoint_decode(b, rows, cols)
    dy = rounded(normal(rows + 1, rows, n) * 0.1, BF16)
    ck, d = Checkpoint(rows, cols, torch.from_numpy(b).cuda()), dev(dy, BF16, pad)
    dw = torch.zeros((cols, n), device="cuda")
    stuck.weight_grad(ck, d, dw)
    refused(_lib.FG_ETIMEOUT, stuck.sync)
    stuck.sync()                      # the error word was cleared
    ref = OT.weight_grad(h, dy)[0]
    _lib.check(stuck.lib.ts_set_wait_limit(stuck.h, 2_000_000_000, 0))
    for handle in (TrainingOps(), stuck):
        dw.fill_(float("nan"))
        handle.weight_grad(ck, d, dw)
        handle.sync()
        # the bound of every weight gradient here: products are exact, each of
        # rows + 8 additions is off by 2^-23 of its partial sum at most
        within(dw, ref, 2.0 ** -23 * (rows + 8) * (np.abs(h).T @ np.abs(dy)) + 1e-30)


def test_wait_limit_refusals(ops):  # noqa: F811
    E = _lib.FG_EINVAL
    refused(E, TrainingOps, 0, wait_limit_ns=0)
    refused(E, TrainingOps, 0, wait_limit_ns=-5)
    refused(E, TrainingOps, 0, flags=1)
    assert ops.lib.ts_set_wait_limit(None, 1, 0) == E


# ---- loops that run more than once ---------------------------------------------------


def device_rows(seed, rows, cols, dtype, scale=1.0, shift=0.0):
    """A matrix made and held on the GPU, and the same in 64 bits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((rows, cols), generator=gen, device="cuda") * scale + shift).to(dtype)
    return x, x.double()


def device_close(got, ref, tol):
    """close(), on the GPU."""
    err = (got.double() - ref).abs() / torch.maximum(ref.abs(), ref.square().mean().sqrt())
    assert err.max().item() <= tol, err.max().item()


# several rows to every resident block, of each number of warps and groups a
# row (8, 16 and 16 warps; a warp to a row), an even and an odd number of them
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("xt, yt", [(F32, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("rows, cols", [(9001, 520), (7000, 1024), (3001, 2048), (2000, 4096), (1501, 5003),
                                        (1000, 8192), (701, 16384), (700, 12000)])
def test_layer_norm_of_many_rows(ops, rows, cols, xt, yt, pad):  # noqa: F811
    x, xd = device_rows(cols, rows, cols, xt, 1.5, 0.4)
    src, y = empty((rows, cols), xt, pad), empty((rows, cols), yt, pad)
    src.copy_(x)
    gamma, beta = vec(normal(1, cols) * 0.1 + 1), vec(normal(2, cols) * 0.1)
    m, r, ck = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), Checkpoint(rows, cols)
    ops.layer_norm(src, gamma, beta, y, m, r, ckpt=ck)
    ops.sync()
    gap_kept(y, pad)
    mean = xd.mean(1)
    d = xd - mean[:, None]
    rstd = (d.square().mean(1) + 1e-5).rsqrt()
    h = d * rstd[:, None]
    # the tolerances of single rows (a few dozen roundings, one more in bf16)
    device_close(y, h * gamma.double() + beta.double(), TOL[yt])
    device_close(m, mean, 1e-5)
    device_close(r, rstd, 1e-5)
    back = torch.empty((rows, cols), device="cuda")
    ops.checkpoint_load(ck, back)
    top = torch.nn.functional.pad(h.abs(), (0, -cols % 32)).unflatten(1, (-1, 32)).amax(2)
    step = torch.exp2(torch.floor(torch.log2(top * (1 + 1e-5))) - 6).repeat_interleave(32, 1)[:, :cols]
    # half a step, a whole one for what 127 steps do not reach, and h's error
    bound = torch.where(h.abs() > 127 * step, step, step / 2) + 2e-5 * h.abs().clamp(min=1)
    assert ((back.double() - h).abs() <= bound).all()


# W = 4, 8, 16 warps a row and G = 2, 32 warps, with even and odd numbers of
# rows a slot: the next rows in flight, both halves of the row sums' buffer
@pytest.mark.parametrize("from_ckpt", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, cols", [(3001, 1000), (2600, 1024), (1900, 2048), (1001, 2048), (1000, 4096),
                                        (609, 4000), (760, 5003), (457, 8192), (700, 12000)])
def test_layer_norm_backward_of_many_rows(ops, rows, cols, dtype, pad, from_ckpt):  # noqa: F811
    x, xd = device_rows(cols, rows, cols, dtype, 1.5, 0.4)
    dy, dyd = device_rows(cols + 1, rows, cols, dtype)
    gamma = vec(normal(1, cols) * 0.1 + 1)
    mean = xd.mean(1).float()
    rstd = ((xd - mean.double()[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    h = (xd - mean.double()[:, None]) * rstd.double()[:, None]
    if from_ckpt:
        src = Checkpoint(rows, cols)
        ops.checkpoint_save(h.float(), src)
        back = torch.empty((rows, cols), device="cuda")
        ops.checkpoint_load(src, back)
        h = back.double()
    else:
        src = empty((rows, cols), dtype, pad)
        src.copy_(x)
    dyt, dx = empty((rows, cols), dtype, pad), empty((rows, cols), dtype, pad)
    dyt.copy_(dy)
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ops.layer_norm_backward(dyt, src, gamma, None if from_ckpt else mean, rstd, dx, dg, db)
    ops.sync()
    gap_kept(dx, pad)
    u = dyd * gamma.double()
    ref = rstd.double()[:, None] * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    device_close(dx, ref, TOL[dtype])
    # at most rows / 8 + 64 additions one after the other, and h is a few
    # roundings off
    n = 2.0 ** -24 * (rows / 8 + 64)
    bound = n * (dyd * h).abs().sum(0) + 2.0 ** -22 * (dyd.abs() * (h.abs() + 1)).sum(0)
    assert ((dg.double() - (dyd * h).sum(0)).abs() <= bound).all()
    assert ((db.double() - dyd.sum(0)).abs() <= n * dyd.abs().sum(0)).all()
    again = torch.empty_like(dx)
    ops.layer_norm_backward(dyt, src, gamma, None if from_ckpt else mean, rstd, again, dg.clone(), db.clone())
    assert torch.equal(again, dx)


# whole tiles for every pair of CTAs and more tokens than one accumulator
# takes: the running partial in the workspace is written and read back
@pytest.mark.parametrize("affine, accumulate", [(False, False), (True, False), (True, True), (False, True)])
@pytest.mark.parametrize("rows, cols, n, pad", [(2304, 2560, 2304, 0), (2433, 2816, 2200, 0), (2304, 2560, 2303, 1),
                                                (8192, 2560, 2048, 0), (4200, 5003, 2050, 2)])
def test_weight_grad_of_many_tokens(ops, rows, cols, n, pad, affine, accumulate):  # noqa: F811
    x, _ = device_rows(rows, rows, cols, F32)
    ck, h = Checkpoint(rows, cols), torch.empty((rows, cols), device="cuda")
    ops.checkpoint_save(x, ck)
    ops.checkpoint_load(ck, h)
    dy, dyd = device_rows(rows + 1, rows, n, BF16, 0.1)
    dyt, dw, db = empty((rows, n), BF16, pad), empty((cols, n), F32, pad), torch.empty(n, device="cuda")
    dyt.copy_(dy)
    old, _ = device_rows(5, cols, n, F32)
    dw.copy_(old)
    more = {"db": db}
    hd = h.double()
    if affine:
        more |= {"gamma": vec(normal(1, cols) * 0.1 + 1), "beta": vec(normal(2, cols) * 0.1)}
        hd = hd * more["gamma"].double() + more["beta"].double()
    db.fill_(3.0)
    ops.weight_grad(ck, dyt, dw, accumulate=accumulate, **more)
    ops.sync()
    gap_kept(dw, pad)
    ref = hd.t() @ dyd
    err = dw.double() - ref
    if accumulate:
        err -= old.double()
    # every addition is off by 2^-23 of its partial sum at most
    size = hd.abs().t() @ dyd.abs() + (old.double().abs() if accumulate else 0)
    assert (err.abs() <= 2.0 ** -23 * (rows + 8) * size).all()
    # the tensor core truncates as it adds, so an accumulator's error grows with
    # its additions: 2.8e-6 of the norm for 8192 tokens in one, a quarter of that
    # for the 2048 that one takes.  Half way: 1.4e-6 (and the addition to dw)
    norm = ref.norm() + (0.1 * old.double().norm() if accumulate else 0)
    assert err.norm() <= 1.4e-6 * norm, (err.norm() / norm).item()
    want = dyd.sum(0) + (3.0 if accumulate else 0)
    assert ((db.double() - want).abs() <= 2.0 ** -24 * (rows / 8 + 64) * (dyd.abs().sum(0) + 3)).all()
    kept, keptb = dw.clone(), db.clone()
    dw.copy_(old)
    db.fill_(3.0)
    ops.weight_grad(ck, dyt, dw, accumulate=accumulate, **more)
    assert torch.equal(dw, kept) and torch.equal(db, keptb)
