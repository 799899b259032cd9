"""GPU parity of the vocabulary operators (embedding and its gradient, the cross
entropy of a linear layer and its gradients) against 64 bits, at the sizes,
strides, types and masks where they can go wrong."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import FgError, TrainingOps, _lib, linear_cross_entropy_workspace
from oracle import training as OT

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}   # one rounding, relative to the value


@pytest.fixture(scope="module")
def ops():
    return TrainingOps(workspace_bytes=256 << 20)


def matrix(a, dtype=F32, pad=0, shift=0):
    """A matrix on the GPU whose rows lie `pad` elements further apart, `shift`
    elements behind an aligned address; what lies between holds NaN."""
    a = torch.as_tensor(a)
    rows, cols = a.shape
    buf = torch.full((rows * (cols + pad) + shift + pad,), float("nan"), dtype=dtype, device="cuda")
    out = torch.as_strided(buf, (rows, cols), (cols + pad, 1), shift)
    return out.copy_(a)


def output(rows, cols, dtype=F32, pad=0, shift=0, fill=-77.0):
    buf = torch.full((rows * (cols + pad) + shift + pad,), fill, dtype=dtype, device="cuda")
    return torch.as_strided(buf, (rows, cols), (cols + pad, 1), shift)


def gap_kept(t, pad, shift, fill=-77.0):
    rows, cols = t.shape
    whole = torch.as_strided(t, (t.untyped_storage().nbytes() // t.element_size(),), (1,), 0)
    keep = torch.ones_like(whole, dtype=torch.bool)
    torch.as_strided(keep, (rows, cols), (cols + pad, 1), shift).fill_(False)
    assert (whole[keep] == fill).all()


def normal(seed, *shape, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale


def tokens(seed, rows, vocab, kind="mixed"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((rows,), vocab // 2)
    if kind == "none":
        return torch.full((rows,), -1)
    ids = (torch.rand(rows, generator=g).pow(3) * vocab).long()   # a few ids often, many seldom
    if kind == "mixed":
        drop = torch.rand(rows, generator=g)
        ids = torch.where(drop < 0.1, torch.tensor(-1), torch.where(drop > 0.95, torch.tensor(vocab), ids))
        ids[torch.rand(rows, generator=g) < 0.01] = 2 ** 40 + 1
    return ids


def within(got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape
    assert torch.equal(got.isnan(), ref.isnan())
    d = torch.where(ref.isfinite(), (got - ref).abs() - bound, torch.where(ref.isnan() | (got == ref), -1.0, 1.0))
    assert (d <= 0).all(), d.max().item()


# ---- embedding -------------------------------------------------------------------

LAYOUTS = [(0, 0), (8, 0), (3, 1)]


@pytest.mark.parametrize("pad, shift", LAYOUTS)
@pytest.mark.parametrize("tt, yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows, cols, vocab", [(1, 1, 1), (1, 1024, 50), (5, 17, 3), (64, 256, 4000), (33, 1003, 100),
                                               (2000, 1032, 777), (300, 5003, 64), (2, 70001, 3)])
def test_embedding(ops, rows, cols, vocab, tt, yt, pad, shift):
    ids = tokens(rows, rows, vocab).cuda()
    table = matrix(normal(1, vocab, cols), tt, pad, shift)
    y = output(rows, cols, yt, pad, shift)
    ops.embedding(ids, table, y, scale=1.7)
    ops.sync()
    gap_kept(y, pad, shift)
    inside = (ids >= 0) & (ids < vocab)
    ref = torch.where(inside[:, None], table.double()[ids.where(inside, torch.tensor(0).cuda())] * 1.7, 0.0)
    # 1.7 and the product are rounded to float32, the result to y's type
    within(y, ref, (2.0 ** -22 + HALF[yt]) * ref.abs())
    assert (y[~inside] == 0).all()


def test_embedding_row_of_no_finite_value_stays_where_it_is(ops):
    table = normal(2, 9, 40).cuda()
    table[4] = float("nan")
    table[5] = float("inf")
    y = output(5, 40)
    ops.embedding(torch.tensor([3, 4, 5, -1, 6]).cuda(), table, y, scale=0.5)
    assert y[1].isnan().all() and (y[2] == float("inf")).all() and y[[0, 3, 4]].isfinite().all()


# one token; one block's sort, with every number of rounds a warp has; several
# tiles; one, two and three passes; a chunk, several, and many of one id
BACK = [(1, 1, 1, "plain"), (1, 300, 5, "none"), (7, 17, 3, "mixed"), (64, 256, 100, "mixed"), (512, 256, 4000, "plain"),
        (1025, 33, 600, "mixed"), (1000, 1003, 70, "mixed"), (5000, 264, 50001, "mixed"), (8192, 40, 131072, "plain"),
        (8193, 64, 300, "mixed"), (20000, 72, 131072, "mixed"), (30001, 40, 1000000, "mixed"), (3000, 520, 9, "one"),
        (40000, 32, 100, "one"), (9000, 24, 77, "none"),
        (65536, 16, 50001, "mixed"), (65537, 16, 70000, "mixed"), (300001, 8, 131072, "mixed"), (300000, 8, 400, "plain"), (700, 5003, 513, "plain"), (3, 70001, 4, "mixed")]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("pad, shift", LAYOUTS)
@pytest.mark.parametrize("dt, tt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows, cols, vocab, kind", BACK)
def test_embedding_backward(ops, rows, cols, vocab, kind, dt, tt, pad, shift, accumulate):
    ids = tokens(rows, rows, vocab, kind).cuda()
    dy = matrix(normal(1, rows, cols), dt, pad, shift)
    inside = (ids >= 0) & (ids < vocab)
    dy[~inside] = float("nan")   # not read
    old = matrix(normal(2, vocab, cols), tt) if accumulate else None
    d = output(vocab, cols, tt, pad, shift)
    if accumulate:
        d.copy_(old)
    ops.embedding_backward(ids, dy, d, scale=1.7, accumulate=accumulate)
    ops.sync()
    gap_kept(d, pad, shift)
    at, src = ids[inside], dy[inside].double()
    ref = torch.zeros((vocab, cols), dtype=torch.float64, device="cuda").index_add_(0, at, src) * 1.7
    size = torch.zeros_like(ref).index_add_(0, at, src.abs()) * 1.7
    n = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    if accumulate:
        ref += old.double()
        size += old.double().abs()
    # n additions, the scale's rounding, the product's and the last sum's
    bound = (n[:, None] + 4) * 2.0 ** -24 * size
    within(d, ref, bound + HALF[tt] * (ref.abs() + bound))
    unused = n == 0
    assert torch.equal(d[unused], old[unused] if accumulate else torch.zeros_like(d[unused]))
    # the same again, to the bit
    again = output(vocab, cols, tt, pad, shift)
    if accumulate:
        again.copy_(old)
    ops.embedding_backward(ids, dy, again, scale=1.7, accumulate=accumulate)
    assert torch.equal(again, d)


def test_embedding_backward_of_no_tokens(ops):
    ids, dy = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty((0, 40), device="cuda")
    d = output(1000, 40)
    ops.embedding_backward(ids, dy, d, accumulate=True)
    assert (d == -77).all()
    ops.embedding_backward(ids, dy, d)
    assert (d == 0).all()
    ops.embedding(ids, d, output(0, 40))
    ops.sync()


def test_embedding_backward_in_a_small_workspace():
    # room for few partials, so that a chunk holds many tokens
    small = TrainingOps(workspace_bytes=1 << 20)
    rows, cols, vocab = 30000, 5000, 50
    ids, dy = tokens(3, rows, vocab, "plain").cuda(), normal(4, rows, cols).cuda()
    d = output(vocab, cols)
    small.embedding_backward(ids, dy, d)
    ref = torch.zeros((vocab, cols), dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
    size = torch.zeros_like(ref).index_add_(0, ids, dy.double().abs())
    within(d, ref, (rows + 2) * 2.0 ** -24 * size)
    with pytest.raises(FgError) as e:
        small.embedding_backward(torch.zeros(300000, dtype=torch.int64, device="cuda"), torch.zeros((300000, 1), device="cuda"),
                                 output(5, 1))
    assert e.value.status == _lib.FG_EUNSUPPORTED


# ---- cross entropy of a linear layer -----------------------------------------------


def loss_bounds(x, w, lse):
    """How far a logit and lse may be off: every addition of the product by
    2^-23 of its partial sum (the tensor core truncates); lse by that, by an
    exponential's 2^-22 and argument, by about 60 + vocab / 1024 additions one
    after the other, and by its own roundings."""
    cols, vocab = x.shape[1], w.shape[0]
    logit = 2.0 ** -23 * (cols + 8) * (x.abs() @ w.abs().t())
    return logit, logit.amax(1) + 2.0 ** -20 + 2.0 ** -24 * (60 + vocab / 1024) + 2.0 ** -22 * lse.abs()


# one of each; less than a tile, ragged tiles, more than one slot of K; rows
# of more than a group of tiles; every pair with more than two tiles
# (up to 16 rows of small weights have a kernel of their own: K cut over warps or
# not, more tiles than warps)
LOSS = [(1, 1, 1), (1, 64, 100), (3, 16, 257), (16, 1024, 3000), (17, 1003, 700), (32, 2056, 50), (8, 40, 60001),
        (31, 264, 45000), (33, 130, 5003), (100, 1024, 3000), (256, 128, 256), (257, 64, 511),
        (512, 256, 4000), (1000, 1003, 777), (4500, 96, 2500), (700, 520, 20011)]


@pytest.mark.parametrize("pad, shift", [(None, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("rows, cols, vocab", LOSS)
def test_linear_cross_entropy(ops, rows, cols, vocab, pad, shift):
    pad = -cols % 8 if pad is None else pad   # None: rows on 16 bytes
    x, w = matrix(normal(1, rows, cols), BF16, pad, shift), matrix(normal(2, vocab, cols, scale=2.5 * cols ** -0.5), BF16, pad, shift)
    targets = tokens(3, rows, vocab).cuda()
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ops.linear_cross_entropy(x, w, targets, loss, lse)
    ops.sync()
    xd, wd = x.double(), w.double()
    logits = xd @ wd.t()
    ref = torch.logsumexp(logits, 1)
    lb, sb = loss_bounds(xd, wd, ref)
    within(lse, ref, sb)
    inside = (targets >= 0) & (targets < vocab)
    at = targets.where(inside, torch.tensor(0).cuda())[:, None]
    want = torch.where(inside, ref - logits.gather(1, at)[:, 0], 0.0)
    within(loss, want, torch.where(inside, sb + lb.gather(1, at)[:, 0] + 2.0 ** -23 * ref.abs(), 0.0))
    # either output alone, the same to the bit
    one, other = torch.empty_like(loss), torch.empty_like(lse)
    ops.linear_cross_entropy(x, w, targets, one, None)
    ops.linear_cross_entropy(x, w, None, None, other)
    assert torch.equal(one, loss) and torch.equal(other, lse)


def run_backward(ops, x, w, targets, lse, g, h, dx_t, dw_t, pad, shift, old=None):
    rows, cols, vocab = x.shape[0], x.shape[1], w.shape[0]
    dx, dw = output(rows, cols, dx_t, pad, shift), output(vocab, cols, dw_t, pad, shift)
    if old is not None:
        dw.copy_(old)
    ops.linear_cross_entropy_backward(x, w, targets, lse, g, dx, dw, g_lse=h, accumulate=old is not None)
    ops.sync()
    gap_kept(dx, pad, shift)
    gap_kept(dw, pad, shift)
    return dx, dw


def check_backward(x, w, targets, lse, g, h, dx, dw, old=None):
    rows, cols, vocab = x.shape[0], x.shape[1], w.shape[0]
    inside = (targets >= 0) & (targets < vocab)
    takes = inside if h is None else torch.ones_like(inside)
    xd = torch.where(takes[:, None], x.double(), 0.0)
    wd, lse = w.double(), torch.where(takes, lse.double(), 0.0)
    logits = xd @ wd.t()
    p = torch.exp(logits - lse[:, None])
    g = torch.where(inside, g.double(), 0.0)
    coef = g if h is None else g + h.double()
    d = coef[:, None] * p
    at = targets.where(inside, torch.tensor(0).cuda())[:, None]
    d.scatter_add_(1, at, -g[:, None])
    # p: the logit, lse as a rounded log2, the exponential; d: one rounding to bf16
    lb, _ = loss_bounds(xd, wd, lse)
    off = lb + 2.0 ** -22 * (lse.abs()[:, None] + logits.abs()) + 2.0 ** -20
    derr = (2.0 ** -8 * d.abs() + (1 + 2.0 ** -8) * 2 * off * (coef[:, None] * p).abs()) * takes[:, None] + 1e-37
    for got, ref, size, err, n, was in (
            (dx, d @ wd, d.abs() @ wd.abs(), derr @ wd.abs(), vocab, None),
            (dw, d.t() @ xd, d.abs().t() @ xd.abs(), derr.t() @ xd.abs(), rows, old)):
        if got is None:
            continue
        bound = err + 2.0 ** -23 * (n + 8) * size
        if was is not None:
            ref = ref + was.double()
            bound = bound + 2.0 ** -24 * (ref.abs() + bound)
        within(got, ref, bound + HALF[got.dtype] * (ref.abs() + bound))
    # roundings of d's entries are independent: as a whole the gradients are as
    # far off as that many errors of 2^-8 at most, uniform (1 / sqrt(3)), and
    # their own roundings
    for got, ref, sq, was in ((dx, d @ wd, (d * d) @ (wd * wd), None), (dw, d.t() @ xd, (d * d).t() @ (xd * xd), old)):
        if got is not None:
            ref = ref if was is None else ref + was.double()
            e = (got.double() - ref).norm()
            assert e <= 2.0 ** -8 * sq.sum().sqrt() + HALF[got.dtype] * ref.norm(), e.item()


@pytest.mark.parametrize("dx_t, dw_t, accumulate", [(BF16, BF16, False), (F32, F32, False), (BF16, F32, True),
                                                    (F32, BF16, True)])
@pytest.mark.parametrize("pad, shift", [(None, 0), (3, 1)])
@pytest.mark.parametrize("rows, cols, vocab", LOSS)
def test_linear_cross_entropy_backward(ops, rows, cols, vocab, pad, shift, dx_t, dw_t, accumulate):
    pad = -cols % 8 if pad is None else pad
    x, w = matrix(normal(1, rows, cols), BF16, pad, shift), matrix(normal(2, vocab, cols, scale=2.5 * cols ** -0.5), BF16, pad, shift)
    targets = tokens(3, rows, vocab).cuda()
    lse = torch.logsumexp(x.double() @ w.double().t(), 1).float()
    g, h = (normal(4, rows) / rows).cuda(), (normal(5, rows) / rows).cuda() if accumulate else None
    if h is None:
        x[(targets < 0) | (targets >= vocab)] = float("nan")   # unscored rows may hold anything
        lse[(targets < 0) | (targets >= vocab)] = float("nan")
    old = matrix(normal(6, vocab, cols, scale=1e-3), dw_t) if accumulate else None
    dx, dw = run_backward(ops, x, w, targets, lse, g, h, dx_t, dw_t, pad, shift, old)
    check_backward(x, w, targets, lse, g, h, dx, dw, old)
    if h is None:
        assert (dx[(targets < 0) | (targets >= vocab)] == 0).all()
    again = run_backward(ops, x, w, targets, lse, g, h, dx_t, dw_t, pad, shift, old)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    # either gradient alone
    alone = output(rows, cols, dx_t, pad, shift)
    ops.linear_cross_entropy_backward(x, w, targets, lse, g, alone, None, g_lse=h)
    assert torch.equal(alone, dx)
    alone = output(vocab, cols, dw_t, pad, shift)
    if old is not None:
        alone.copy_(old)
    ops.linear_cross_entropy_backward(x, w, targets, lse, g, None, alone, g_lse=h, accumulate=accumulate)
    assert torch.equal(alone, dw)
    ops.linear_cross_entropy_backward(x, w, targets, lse, g, None, None, g_lse=h)


# several pieces of the vocabulary (dx is summed over them, cut or not), several
# blocks of rows, copies of unaligned rows by pieces
@pytest.mark.parametrize("pad, shift", [(0, 0), (3, 1)])
@pytest.mark.parametrize("rows, cols, vocab", [(300, 256, 5000), (1500, 64, 2500), (40, 512, 9000), (20, 200, 20000)])
def test_linear_cross_entropy_in_a_small_workspace(rows, cols, vocab, pad, shift):
    x, w = matrix(normal(1, rows, cols), BF16, pad, shift), matrix(normal(2, vocab, cols, scale=2.5 * cols ** -0.5), BF16, pad, shift)
    targets = tokens(3, rows, vocab).cuda()
    least, most = linear_cross_entropy_workspace(rows, cols, vocab)
    lse = torch.logsumexp(x.double() @ w.double().t(), 1).float()
    g = (normal(4, rows) / rows).cuda()
    for size in sorted({max(1 << 20, least), max(1 << 20, (3 * least + most) // 4), max(1 << 20, (least + most) // 2)}):
        ops = TrainingOps(workspace_bytes=size)
        loss, got = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ops.linear_cross_entropy(x, w, targets, loss, got)
        logits = x.double() @ w.double().t()
        ref = torch.logsumexp(logits, 1)
        within(got, ref, loss_bounds(x.double(), w.double(), ref)[1])
        for old in (None, matrix(normal(6, vocab, cols, scale=1e-3), F32)):
            dx, dw = run_backward(ops, x, w, targets, lse, g, None, BF16, F32, pad, shift, old)
            check_backward(x, w, targets, lse, g, None, dx, dw, old)


def test_linear_cross_entropy_workspace_too_small():
    rows, cols, vocab = 3000, 1024, 500
    least, most = linear_cross_entropy_workspace(rows, cols, vocab)
    assert least < most
    ops = TrainingOps(workspace_bytes=1 << 20)
    x, w = torch.zeros((rows, cols), dtype=BF16, device="cuda"), torch.zeros((vocab, cols), dtype=BF16, device="cuda")
    v, t = torch.zeros(rows, device="cuda"), torch.zeros(rows, dtype=torch.int64, device="cuda")
    with pytest.raises(FgError) as e:
        ops.linear_cross_entropy_backward(x, w, t, v, v, torch.empty_like(x), torch.empty_like(w))
    assert e.value.status == _lib.FG_EUNSUPPORTED


def test_linear_cross_entropy_of_logits_that_are_not_finite(ops):
    """-inf logits have probability 0; rows of nothing else, NaN and +inf."""
    inf, nan = float("inf"), float("nan")
    rows, cols, vocab = 6, 8, 300
    w = torch.zeros((vocab, cols))
    w[:, 0] = 1.0
    w[:, 1] = torch.arange(vocab) < 7       # -inf logits of the first few for rows with x[1] = -inf
    w[:, 1][w[:, 1] == 0] = 0.0
    x = torch.zeros((rows, cols))
    x[:, 0] = torch.arange(rows) * 0.5
    x[1, 0] = -inf      # every logit -inf
    x[2, 0] = nan
    x[3, 0] = inf
    x[4, 0] = 3e38      # (3e38 is finite in bf16)
    x[4, 1] = 0
    targets = torch.tensor([0, 1, 2, 3, 299, -1])
    # 0 * inf: columns of w that are 0 would give NaN, so x's infinities meet ones
    x[:, 1:] = 0
    w[:, 1:] = 0
    xb, wb = x.to(BF16), w.to(BF16)
    ref_loss, ref_lse = OT.linear_cross_entropy(xb.double().numpy()[:, :1], wb.double().numpy()[:, :1], targets.tolist())
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    xc, wc = xb.cuda()[:, :1], wb.cuda()[:, :1]
    xc, wc = matrix(xc.float(), BF16, 7), matrix(wc.float(), BF16, 7)
    ops.linear_cross_entropy(xc, wc, targets.cuda(), loss, lse)
    ops.sync()
    for got, ref in ((loss, ref_loss), (lse, ref_lse)):
        got = got.double().cpu().numpy()
        for r in (0, 1, 2, 3, 5):
            assert got[r] == ref[r] or (np.isnan(got[r]) and np.isnan(ref[r])) or abs(got[r] - ref[r]) < 1e-5, (r, got, ref)
    # a row of -inf logits takes no gradient, of x's and of w's
    g = torch.full((rows,), 0.25, device="cuda")
    dx, dw = output(rows, 1), output(vocab, 1)
    keep = [0, 1, 5]
    t = targets.cuda()[keep]
    ops.linear_cross_entropy_backward(matrix(xc[keep].float(), BF16, 7), wc, t, lse[keep].contiguous(), g[:3].contiguous(), dx[:3], dw)
    ops.sync()
    rdx, rdw, _ = OT.linear_cross_entropy_backward(xb.double().numpy()[keep][:, :1], wb.double().numpy()[:, :1],
                                                   t.tolist(), lse[keep].double().cpu().numpy(), [0.25] * 3)
    assert (dx[1:3] == 0).all()
    assert np.allclose(dx[:3].cpu().numpy(), rdx, atol=3e-3) and np.allclose(dw.cpu().numpy(), rdw, atol=3e-3)


def test_linear_cross_entropy_of_no_rows(ops):
    x, w = torch.empty((0, 64), dtype=BF16, device="cuda"), torch.ones((300, 64), dtype=BF16, device="cuda")
    t, v = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    ops.linear_cross_entropy(x, w, t, v, v)
    for dtype in (F32, BF16):
        dw = output(300, 64, dtype)
        ops.linear_cross_entropy_backward(x, w, t, v, v, torch.empty_like(x), dw, accumulate=True)
        assert (dw == -77).all()
        ops.linear_cross_entropy_backward(x, w, t, v, v, torch.empty_like(x), dw)
        assert (dw == 0).all()


def test_waits_that_run_out():
    """Without its copies every wait of the product expires, the call reports it
    and the next one is right."""
    ops = TrainingOps(workspace_bytes=8 << 20, wait_limit_ns=1_000_000, flags=_lib.FG_FLAG_INJECT_NO_LOADS)
    rows, cols, vocab = 300, 256, 1000
    x, w = normal(1, rows, cols).cuda().to(BF16), normal(2, vocab, cols, scale=0.1).cuda().to(BF16)
    t = tokens(3, rows, vocab).cuda()
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ref = torch.logsumexp(x.double() @ w.double().t(), 1)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ops.linear_cross_entropy(x, w, t, loss, lse)
    with pytest.raises(FgError) as e:
        ops.sync()
    assert e.value.status == _lib.FG_ETIMEOUT
    ops.linear_cross_entropy_backward(x, w, t, ref.float(), loss, dx, dw)
    with pytest.raises(FgError) as e:
        ops.sync()
    assert e.value.status == _lib.FG_ETIMEOUT
    _lib.check(ops.lib.ts_set_wait_limit(ops.h, 2_000_000_000, 0))
    ops.linear_cross_entropy(x, w, t, loss, lse)
    ops.sync()
    within(lse, ref, loss_bounds(x.double(), w.double(), ref)[1])


# ---- together ------------------------------------------------------------------------


def step(ops, ids, targets, table, x, loss, lse, g, dx, dw):
    """Tied weights: the embedding, the loss on it, and the table's gradient from both."""
    ops.embedding(ids, table, x, scale=2.0)
    ops.linear_cross_entropy(x, table, targets, loss, lse)
    ops.linear_cross_entropy_backward(x, table, targets, lse, g, dx, dw)
    ops.embedding_backward(ids, dx, dw, scale=2.0, accumulate=True)


def tied(rows=700, cols=264, vocab=3001):
    table = normal(1, vocab, cols, scale=0.3).cuda().to(BF16)
    ids, targets = tokens(2, rows, vocab).cuda(), tokens(3, rows, vocab).cuda()
    f = dict(device="cuda")
    return [ids, targets, table, torch.empty((rows, cols), dtype=BF16, **f), torch.empty(rows, **f), torch.empty(rows, **f),
            torch.full((rows,), 1.0 / rows, **f), torch.empty((rows, cols), **f), torch.empty((vocab, cols), **f)]


def test_tied_step(ops):
    a = tied()
    step(ops, *a)
    ops.sync()
    ids, targets, table, x, loss, lse, g, dx, dw = a
    inside = (ids >= 0) & (ids < len(table))
    check_backward(x, table, targets, lse, g, None, dx, None)
    part = torch.empty_like(dw)
    ops.linear_cross_entropy_backward(x, table, targets, lse, g, None, part)
    want = part.double().index_add(0, ids[inside], dx[inside].double() * 2.0)
    size = part.double().abs().index_add(0, ids[inside], dx[inside].double().abs() * 2.0)
    within(dw, want, 2.0 ** -24 * (len(ids) + 4) * size)


# every kernel that a call's size chooses: few rows of a small table, few tokens,
# a cluster's sort, a sort of several launches
SIZES = [(9, 264, 3001), (700, 264, 3001), (3000, 72, 3001), (20000, 40, 3001)]


@pytest.mark.parametrize("rows, cols, vocab", SIZES)
def test_captured_and_replayed(ops, rows, cols, vocab):
    a, b = tied(rows, cols, vocab), tied(rows, cols, vocab)
    step(ops, *a)
    mine = TrainingOps(workspace_bytes=256 << 20)   # (as `ops`: sums are cut by what it holds)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(mine, *b)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step(mine, *b)
    for _ in range(2):
        for t in b[3:6] + b[7:]:
            t.fill_(float("nan"))
        graph.replay()
        mine.sync()
        for s, t in zip(a, b):
            assert torch.equal(s, t)
    # other tokens in the same buffers
    b[0].copy_(tokens(9, len(b[0]), len(b[2])).cuda())
    a[0].copy_(b[0])
    graph.replay()
    step(ops, *a)
    mine.sync()
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("rows, cols, vocab", SIZES)
def test_two_handles_on_two_streams(rows, cols, vocab):
    ref, runs = tied(rows, cols, vocab), [tied(rows, cols, vocab), tied(rows, cols, vocab)]
    handles = [TrainingOps(workspace_bytes=64 << 20) for _ in range(3)]
    step(handles[2], *ref)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for o, s, r in zip(handles, streams, runs):
            with torch.cuda.stream(s):
                step(o, *r)
    torch.cuda.synchronize()
    for r in runs:
        for x, y in zip(ref, r):
            assert torch.equal(x, y)


def test_calls_of_one_handle_in_any_order(ops):
    """Calls of different sizes follow each other in one workspace, nothing
    waited for: each finds what it needs as it was meant to be."""
    want = [tied(*s) for s in SIZES]
    fresh = TrainingOps(workspace_bytes=256 << 20)
    for a in want:
        step(fresh, *a)
        fresh.sync()
    got = [tied(*s) for s in SIZES]
    for i in (0, 3, 1, 0, 2, 3, 0, 1, 2, 2, 0, 3):
        step(ops, *got[i])
    ops.sync()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_loss_gradient_is_the_differences(ops):
    """Along a direction of x and of w, in steps that bf16 holds exactly."""
    rows, cols, vocab = 40, 64, 500
    x, w = torch.round(normal(1, rows, cols) * 8) / 8, torch.round(normal(2, vocab, cols) * 8) / 32
    targets, g = tokens(3, rows, vocab).cuda(), (normal(4, rows).abs() + 0.5).cuda()

    def total(x, w):
        loss = torch.empty(rows, device="cuda")
        ops.linear_cross_entropy(x.cuda().to(BF16), w.cuda().to(BF16), targets, loss, None)
        return (loss.double() * g.double()).sum().item()

    lse = torch.empty(rows, device="cuda")
    xb, wb = x.cuda().to(BF16), w.cuda().to(BF16)
    ops.linear_cross_entropy(xb, wb, targets, None, lse)
    dx, dw = output(rows, cols), output(vocab, cols)
    ops.linear_cross_entropy_backward(xb, wb, targets, lse, g, dx, dw)
    # x, w and the steps are multiples of 2^-7 below 2: exact in bf16.  The second
    # difference's term is bounded by the step's square times the logits' spread
    step = 2.0 ** -7
    for t, d, at in ((x, dx, 0), (w, dw, 1)):
        u = torch.sign(normal(5 + at, *t.shape)) * (normal(7 + at, *t.shape).abs() > 1.5)
        keep = ((t + step * u).to(BF16).float() == t + step * u) & ((t - step * u).to(BF16).float() == t - step * u)
        u = u * keep
        up, down = ((total(t + s * step * u, w) if at == 0 else total(x, t + s * step * u)) for s in (1, -1))
        along = (d.cpu().double() * u.double()).sum().item()
        # third derivatives of a log-sum-exp along a direction: the cube of the
        # logits' change, and float32 losses of about 5 in both sums
        delta = (step * (u @ w.t() if at == 0 else x @ u.t())).abs().amax(1).double()
        bound = (delta ** 3 * g.cpu().double()).sum().item() / step + 2 * 2.0 ** -20 * 5 * g.sum().item() / step
        bound += 2.0 ** -8 * (d.cpu().double().abs() * u.double().abs()).sum().item()
        assert abs((up - down) / (2 * step) - along) <= bound, (up - down, along, bound)


def test_offsets_past_32_bits():
    """Tables of more than 2^31 elements, looked at near their ends."""
    ops = TrainingOps(workspace_bytes=512 << 20)
    vocab, cols, rows = 1 << 20, 2064, 40
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.empty((vocab, cols), dtype=BF16, device="cuda")
    for part in w.split(1 << 17):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * 2.5 * cols ** -0.5)
    ids = torch.cat([torch.arange(vocab - 30, vocab), torch.arange(10) * 100003]).cuda()
    x = output(rows, cols, BF16)
    ops.embedding(ids, w, x)
    assert torch.equal(x, w[ids])
    x.mul_(0.5)
    loss, lse, grad = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.full((rows,), 0.1, device="cuda")
    ops.linear_cross_entropy(x, w, ids, loss, lse)
    logits = torch.cat([x.double() @ part.double().t() for part in w.split(1 << 17)], 1)
    ref = torch.logsumexp(logits, 1)
    tail = slice(vocab - 4096, vocab)
    bound = 2.0 ** -23 * (cols + 8) * x.double().abs().sum(1) * w.abs().max().double() + 2.0 ** -20 + 2.0 ** -24 * 2000 + 2.0 ** -22 * ref
    within(lse, ref, bound)
    dx, dw = output(rows, cols), torch.full_like(w, 7.0)
    ops.linear_cross_entropy_backward(x, w, ids, lse, grad, dx, dw)
    ops.sync()
    d = 0.1 * torch.exp(logits - lse.double()[:, None])
    d.scatter_add_(1, ids[:, None], torch.full((rows, 1), -0.1, dtype=torch.float64, device="cuda"))
    want = d[:, tail].t() @ x.double()
    e = (dw[tail].double() - want).norm()
    # d's roundings and dw's own: 2^-8 of each, at most
    assert e <= 2 * 2.0 ** -8 * want.norm(), e
    back = torch.full_like(w, 7.0)
    ops.embedding_backward(ids, dx, back)
    ops.sync()
    assert torch.equal(back[ids], dx.to(BF16))   # (each id once)
    assert (back[vocab - 5000:vocab - 30] == 0).all() and (back[:100000][1:] == 0).all()


# ---- refusals -----------------------------------------------------------------------------


def test_refusals(ops):
    x, w = torch.zeros((4, 64), dtype=BF16, device="cuda"), torch.zeros((9, 64), dtype=BF16, device="cuda")
    t, v = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    bad = [
        (lambda: ops.linear_cross_entropy(x.float(), w, t, v, v), _lib.FG_EINVAL),
        (lambda: ops.linear_cross_entropy(x, w.float(), t, v, v), _lib.FG_EINVAL),
        (lambda: ops.linear_cross_entropy(x, w[:, :32], t, v, v), _lib.FG_ESHAPE),
        (lambda: ops.linear_cross_entropy(x, w, t[:3], v, v), _lib.FG_ESHAPE),
        (lambda: ops.linear_cross_entropy(x, w, t.int(), v, v), _lib.FG_EINVAL),
        (lambda: ops.linear_cross_entropy(x, w, None, v, v), _lib.FG_EINVAL),
        (lambda: ops.linear_cross_entropy(x, w[:0], t, v, v), _lib.FG_ESHAPE),
        (lambda: ops.linear_cross_entropy_backward(x, w, t, None, v, x, w), _lib.FG_EINVAL),
        (lambda: ops.linear_cross_entropy_backward(x, w, t, v, None, x, w), _lib.FG_EINVAL),
        (lambda: ops.linear_cross_entropy_backward(x, w, t, v, v, x.half(), w), _lib.FG_EINVAL),
        (lambda: ops.linear_cross_entropy_backward(x, w, t, v, v, x, w[:5]), _lib.FG_ESHAPE),
        (lambda: ops.embedding(t, w, x[:3]), _lib.FG_ESHAPE),
        (lambda: ops.embedding(t.int(), w, x), _lib.FG_EINVAL),
        (lambda: ops.embedding(t, w.cpu(), x), _lib.FG_EINVAL),
        (lambda: ops.embedding(t, w.t(), x), _lib.FG_ESHAPE),
        (lambda: ops.embedding_backward(t, x, w[:, :32]), _lib.FG_ESHAPE),
        (lambda: ops.embedding_backward(t, x, w[:0]), _lib.FG_ESHAPE),
    ]
    for f, status in bad:
        with pytest.raises(FgError) as e:
            f()
        assert e.value.status == status
