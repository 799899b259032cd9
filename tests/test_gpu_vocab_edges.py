"""GPU tests of the vocabulary operators where 32 bits or the workspace end: logits
near float32's largest value and rows that hold both ends, losses far smaller than
their logits, sums longer than one accumulator takes, how a workspace cuts a call,
and outputs in place of inputs."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

from group_execution_gb300 import FgError, TrainingOps, _lib, linear_cross_entropy_workspace
from tests.test_gpu_vocab import check_backward, matrix, normal, output, run_backward, tied, tokens, within

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def ops():
    return TrainingOps(workspace_bytes=256 << 20)


# ---- logits at float32's ends --------------------------------------------------------

# rows whose kernel takes K from registers, in one part and in many; tiles: a ragged
# one, several of them, rows of more than one
SIZES = [(7, 300), (14, 60001), (40, 300), (300, 1777)]


def ends(rows, vocab, masked):
    """x and w of one column: rows of logits 0.5 to 3; of NaN; of +inf; of values
    near the largest float32, two of them or (masked) -inf beside them; and,
    where no weight is -inf, of -inf alone."""
    w = torch.where(torch.arange(vocab) % 3 == 0, 0.5, 1.0)[:, None]
    if masked:
        w[torch.arange(vocab) % 5 == 2] = -INF
    values = [1.0, NAN, INF, 3e38, 3.0] + ([] if masked else [-INF, -3e38])
    x = torch.tensor([values[i % len(values)] for i in range(rows)])[:, None]
    return matrix(x, BF16, 7), matrix(w, BF16, 7)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rows, vocab", SIZES)
def test_logits_at_the_ends_of_float32(ops, rows, vocab, masked):
    x, w = ends(rows, vocab, masked)
    targets = (torch.arange(rows) * 7 % vocab).cuda()
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ops.linear_cross_entropy(x, w, targets, loss, lse)
    ops.sync()
    logits = x.double() @ w.double().t()   # (one product each: exact)
    ref = torch.logsumexp(logits, 1)
    ref[(logits == INF).any(1)] = NAN
    # the exponentials and their argument, about 60 + vocab / 1024 additions, the logarithm and lse's rounding
    error = 2.0 ** -20 + 2.0 ** -24 * (60 + vocab / 1024)
    within(lse, ref, error + 2.0 ** -23 * ref.abs())
    at = logits.gather(1, targets[:, None])
    want = torch.logsumexp(logits - at, 1)   # (lse - logit would lose a small loss in 64 bits too)
    want[(at == -INF)[:, 0]] = INF
    want[ref.isnan()] = NAN
    within(loss, want, error + 2.0 ** -23 * want.abs())


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rows, vocab", SIZES)
def test_gradient_of_logits_at_the_ends_of_float32(ops, rows, vocab, masked):
    x, w = ends(rows, vocab, masked)
    logits = x.double() @ w.double().t()
    lse = torch.logsumexp(logits, 1).float()
    g = ((0.25 + torch.arange(rows) % 3 * 0.5) / 1024).cuda()
    targets = (torch.arange(rows) * 7 % vocab).cuda()
    bad = logits.isnan().any(1) | (logits == INF).any(1)
    targets[bad] = -1                                        # not scored: may hold anything
    dx, dw = output(rows, 1), output(vocab, 1)
    ops.linear_cross_entropy_backward(x, w, targets, lse, g, dx, dw)
    ops.sync()
    takes = ~bad & (lse != -INF)
    d = torch.exp(logits - lse.double()[:, None]) * g.double()[:, None]
    d[takes] = d[takes].scatter_add(1, targets[takes][:, None], -g[takes].double()[:, None])
    d[~takes] = 0.0
    # an exponential's 2^-20 and one rounding to bf16, the sums' additions
    off = 2.0 ** -8 * d.abs() + 2.0 ** -19 * g.double()[:, None] + 1e-37
    off[~takes] = 0.0
    xd = torch.where(takes[:, None], x.double(), 0.0)
    within(dw, d.t() @ xd, off.t() @ xd.abs() + 2.0 ** -23 * (rows + 8) * (d.abs().t() @ xd.abs()))
    if not masked:   # (0 * -inf is NaN in dx)
        wd = w.double()
        within(dx, d @ wd, off @ wd.abs() + 2.0 ** -23 * (vocab + 8) * (d.abs() @ wd.abs()))
        assert (dx[~takes] == 0).all()


# ---- losses that are small beside their logits -----------------------------------------


@pytest.mark.parametrize("far", [40.0, 8.0])
@pytest.mark.parametrize("rows, vocab", [(1, 3000), (16, 40001), (60, 3000), (300, 20011)])
def test_loss_of_confident_rows(ops, rows, vocab, far):
    """The target's logit is a, the others' are far below: the loss is as near to
    its value whatever a is, and never negative."""
    a = torch.arange(rows) % 30 * 4.0 + 4.0
    a[rows // 2:] *= 256.0
    c = -far + torch.arange(vocab) % 8 * 0.25                # (of eight bits, like a: exact in bf16, a + c in float32)
    t = vocab // 3
    c[t] = 0.0
    x = matrix(torch.stack([a, torch.ones(rows)], 1), BF16, 6)
    w = matrix(torch.stack([torch.ones(vocab), c], 1), BF16, 6)
    targets = torch.full((rows,), t).cuda()
    targets[rows // 4] = 0                                   # one that is not its row's largest
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ops.linear_cross_entropy(x, w, targets, loss, lse)
    ops.sync()
    rest = torch.exp(c.double().cuda()).sum() - 1.0          # beside the target's 1
    want = torch.log1p(rest) - c.double().cuda()[targets]
    # the others' exponentials and arguments, about 60 + vocab / 1024 additions, the
    # logarithm's and the loss's roundings
    error = 2.0 ** -20 * rest / (1 + rest) + 2.0 ** -24 * (60 + vocab / 1024) + 2.0 ** -22 * torch.log1p(rest)
    within(loss, want, error + 2.0 ** -24 * want)
    assert (loss >= 0).all()
    within(lse, a.double().cuda() + torch.log1p(rest), error + 2.0 ** -24 * (a.double().cuda() + 1))


@pytest.mark.parametrize("rows, cols, vocab", [(40, 8192, 300), (300, 2056, 5003), (9, 8192, 300)])
def test_gradient_of_confident_rows(ops, rows, cols, vocab):
    """The target's logit is a sum of one sign, far above the others: whatever the
    tensor core loses of it, the gradient is that of the loss, here nothing."""
    gen = torch.Generator().manual_seed(0)
    x = matrix(1 + torch.rand((rows, cols), generator=gen), BF16, -cols % 8)
    w = torch.zeros((vocab, cols))
    w[vocab // 3] = (1 + torch.rand(cols, generator=gen)) * (40 / 2.25 / cols)
    w = matrix(w, BF16, -cols % 8)
    targets = torch.full((rows,), vocab // 3).cuda()
    loss, lse, g = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.ones(rows, device="cuda")
    ops.linear_cross_entropy(x, w, targets, loss, lse)
    dx, dw = output(rows, cols), output(vocab, cols)
    ops.linear_cross_entropy_backward(x, w, targets, lse, g, dx, dw)
    ops.sync()
    xd, wd = x.double(), w.double()
    d = torch.softmax(xd @ wd.t(), 1)
    d[:, vocab // 3] -= 1.0
    # of d: lse's rounding at its size and an exponential's 2^-21, and one rounding to bf16
    off = 2.0 ** -8 * d.abs() + 2.0 ** -21 + 2.0 ** -23 * lse.double()[:, None].abs()
    off[:, torch.arange(vocab) != vocab // 3] = 1e-12        # (e^-38 of the others)
    within(dx, d @ wd, off @ wd.abs())
    within(dw, d.t() @ xd, off.t() @ xd.abs())


# ---- sums longer than one accumulator ----------------------------------------------------

# An MMA adds 16 products to its accumulator, and each of the 17 may lose 2^-24 of
# the sum (the tensor core truncates).  An accumulator takes 2048 products, whose
# partial sums are half of the last on average; what accumulators come to is added in
# float32, rounded to nearest.  All terms are of one sign and d is exact in bf16.


def sum_bound(n):
    return 17 * 2.0 ** -24 * (2048 / 16) / 2 + 2.0 ** -24 * (n / 2048 + 4)


def test_weight_gradient_of_many_rows():
    rows, cols, vocab = 1 << 19, 64, 128
    ops = TrainingOps(workspace_bytes=640 << 20)
    x = (1 + torch.rand((rows, cols), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")).to(BF16)
    w = torch.zeros((vocab, cols), dtype=BF16, device="cuda")
    targets = torch.full((rows,), -1, device="cuda")
    lse = torch.full((rows,), vocab, device="cuda").log()
    one = torch.ones(rows, device="cuda")
    dw = output(vocab, cols)
    ops.linear_cross_entropy_backward(x, w, targets, lse, one, None, dw, g_lse=one)
    ops.sync()
    ref = (x.sum(0, dtype=torch.float64) / vocab).expand(vocab, cols)
    within(dw, ref, sum_bound(rows) * ref)


def test_input_gradient_of_a_large_vocabulary():
    # (as many tiles of dx as leave its sums uncut)
    rows, cols, vocab = 4096, 4096, 1 << 19
    ops = TrainingOps(workspace_bytes=5 << 30)
    gen = torch.Generator(device="cuda").manual_seed(0)
    w = torch.empty((vocab, cols), dtype=BF16, device="cuda")
    for part in w.split(1 << 16):
        part.copy_(1 + torch.rand(part.shape, generator=gen, device="cuda"))
    x = torch.zeros((rows, cols), dtype=BF16, device="cuda")
    targets = torch.full((rows,), -1, device="cuda")
    lse = torch.full((rows,), vocab, device="cuda").log()
    one = torch.ones(rows, device="cuda")
    dx = output(rows, cols)
    ops.linear_cross_entropy_backward(x, w, targets, lse, one, dx, None, g_lse=one)
    ops.sync()
    ref = torch.stack([part.sum(0, dtype=torch.float64) for part in w.split(1 << 16)]).sum(0) / vocab
    ref = ref.expand(rows, cols)
    within(dx, ref, sum_bound(vocab) * ref)


# ---- how a workspace cuts a call -----------------------------------------------------------


def launches(call):
    """How many kernels a call launches: the nodes of its captured graph."""
    cu = C.CDLL("libcuda.so.1")
    stream, graph, n = torch.cuda.Stream(), C.c_void_p(), C.c_size_t()
    at = C.c_void_p(stream.cuda_stream)
    torch.cuda.synchronize()
    assert cu.cuStreamBeginCapture_v2(at, 1) == 0
    call(stream.cuda_stream)
    assert cu.cuStreamEndCapture(at, C.byref(graph)) == 0
    assert cu.cuGraphGetNodes(graph, None, C.byref(n)) == 0
    assert cu.cuGraphDestroy(graph) == 0
    return n.value


@pytest.mark.parametrize("rows, cols, vocab", [(64, 1001, 20000), (200, 1003, 50001), (1000, 65, 3001)])
def test_loss_in_the_most_workspace(rows, cols, vocab):
    """What the query calls the most takes all rows and the whole vocabulary at
    once, copies of unaligned rows too: as any larger workspace does."""
    x, w = matrix(normal(1, rows, cols), BF16, 0, 1), matrix(normal(2, vocab, cols, scale=cols ** -0.5), BF16, 0, 1)
    targets = tokens(3, rows, vocab).cuda()
    most = linear_cross_entropy_workspace(rows, cols, vocab)[1]
    got = []
    for size in (most, 8 * most):
        ops = TrainingOps(workspace_bytes=size)
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ops.linear_cross_entropy(x, w, targets, loss, lse)
        ops.sync()
        # the copies of x and w, the products, the join
        assert launches(lambda s: ops.linear_cross_entropy(x, w, targets, loss, lse, stream=s)) == 4
        got.append((loss, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("rows, cols, vocab, before", [(256, 4096, 100, 1), (1000, 1024, 777, 1), (3000, 264, 300, 1),
                                                      (300, 256, 1000, 0)])
def test_copy_of_x_is_no_longer_than_the_logits(ops, rows, cols, vocab, before):
    """dw's copy of x has a launch of its own where the logits are too few to hide it."""
    x, w = matrix(normal(1, rows, cols), BF16), matrix(normal(2, vocab, cols, scale=2.5 * cols ** -0.5), BF16)
    targets = tokens(3, rows, vocab).cuda()
    lse = torch.logsumexp(x.double() @ w.double().t(), 1).float()
    g = (normal(4, rows) / rows).cuda()
    x[(targets < 0) | (targets >= vocab)] = NAN              # unscored rows may hold anything
    dx, dw = run_backward(ops, x, w, targets, lse, g, None, BF16, F32, 0, 0)
    check_backward(x, w, targets, lse, g, None, dx, dw)

    def count(dx, dw):
        return launches(lambda s: ops.linear_cross_entropy_backward(x, w, targets, lse, g, dx, dw, stream=s))
    assert count(dx, dw) == count(dx, None) + before


# ---- outputs in place of inputs --------------------------------------------------------------


@pytest.mark.parametrize("size", [(9, 264, 3001), (700, 264, 3001), (33, 1003, 700)])
def test_input_gradient_in_place(size):
    """dx may be x: with room for the whole vocabulary, and for a piece at a time."""
    rows, cols, vocab = size
    for room in (0, 1):
        ops = TrainingOps(workspace_bytes=max(1 << 20, linear_cross_entropy_workspace(*size)[1 - room]))
        _, targets, w, _, loss, lse, g, _, dw = tied(*size)
        x = normal(4, rows, cols).cuda().to(BF16)
        ops.linear_cross_entropy(x, w, targets, loss, lse)
        dx, dw2 = torch.empty_like(x), torch.empty_like(dw)
        ops.linear_cross_entropy_backward(x, w, targets, lse, g, dx, dw)
        ops.linear_cross_entropy_backward(x, w, targets, lse, g, x, dw2)
        ops.sync()
        assert torch.equal(dx, x) and torch.equal(dw, dw2)


def test_outputs_in_place_of_inputs_are_refused(ops):
    """An output that starts where an input does reaches no kernel, dx on an x of
    its own dtype and pitch aside."""
    buf = torch.zeros(8192, device="cuda")

    def at(rows, cols, dtype, ld):
        return torch.as_strided(buf.view(dtype), (rows, cols), (ld, 1))

    x, w = torch.zeros((4, 64), dtype=BF16, device="cuda"), torch.zeros((9, 64), dtype=BF16, device="cuda")
    ids, v, u = torch.zeros(4, dtype=torch.int64, device="cuda"), *torch.zeros((2, 4), device="cuda")
    xs, ws, vs = at(4, 64, BF16, 64), at(9, 64, BF16, 64), buf[:4]
    ls = buf[:8].view(torch.int64)
    back = ops.linear_cross_entropy_backward
    bad = [
        lambda: ops.embedding(ids, ws, xs),
        lambda: ops.embedding(ids, ws, at(4, 64, F32, 64)),
        lambda: ops.embedding(ls, w, xs),
        lambda: ops.embedding_backward(ids, xs, ws),
        lambda: ops.embedding_backward(ids, xs, at(9, 64, F32, 64)),
        lambda: ops.embedding_backward(ls, x, ws),
        lambda: ops.linear_cross_entropy(xs, w, ids, vs, u),
        lambda: ops.linear_cross_entropy(x, ws, ids, u, vs),
        lambda: ops.linear_cross_entropy(x, w, ls, vs, u),
        lambda: ops.linear_cross_entropy(x, w, ids, vs, vs),
        lambda: back(xs, w, ids, v, v, at(4, 64, BF16, 72), None),
        lambda: back(xs, w, ids, v, v, at(4, 64, F32, 64), None),
        lambda: back(x, ws, ids, v, v, xs, None),
        lambda: back(x, ws, ids, v, v, None, ws),
        lambda: back(xs, w, ids, v, v, None, ws),
        lambda: back(x, w, ids, v, v, xs, ws),
        lambda: back(x, w, ids, vs, v, xs, None),
        lambda: back(x, w, ids, v, vs, None, ws),
        lambda: back(x, w, ids, v, v, None, ws, g_lse=vs),
        lambda: back(x, w, ls, v, v, xs, None),
    ]
    for f in bad:
        with pytest.raises(FgError) as e:
            f()
        assert e.value.status == _lib.FG_EINVAL
    ops.sync()


# ---- values below the smallest normal float32 ---------------------------------------------------


@pytest.mark.parametrize("rows", [40, 3000, 20000])
def test_embedding_gradient_added_to_small_values(ops, rows):
    """A sum that is added in memory may be taken as zero, and left as zero, where
    it is below the smallest normal float32; rows without tokens are kept."""
    cols, vocab, tiny = 40, 5000, 2.0 ** -126
    ids = tokens(1, rows, vocab // 2).cuda()
    dy, old = normal(2, rows, cols).cuda() * tiny, normal(3, vocab, cols).cuda() * tiny
    d = old.clone()
    ops.embedding_backward(ids, dy, d, scale=0.5, accumulate=True)
    ops.sync()
    inside = (ids >= 0) & (ids < vocab)
    at, src = ids[inside], dy[inside].double() * 0.5
    ref = old.double().index_add(0, at, src)
    n = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    size = old.double().abs().index_add(0, at, src.abs())
    # three values of an addition in memory, 2^-126 each; additions among subnormals are exact or round by 2^-150
    within(d, ref, 3 * tiny + (n[:, None] + 4) * 2.0 ** -24 * (size + tiny))
    assert torch.equal(d[n == 0], old[n == 0])


# ---- waits --------------------------------------------------------------------------------------


def test_waits_that_run_out_between_chains():
    """Without its copies every wait of a product over several chains expires, the
    call reports it and the next one is right."""
    ops = TrainingOps(wait_limit_ns=1_000_000, flags=_lib.FG_FLAG_INJECT_NO_LOADS)
    rows, cols, vocab = 2500, 1100, 5000
    x, w = matrix(normal(1, rows, cols), BF16, 4), matrix(normal(2, vocab, cols, scale=0.05), BF16, 4)
    targets = tokens(3, rows, vocab).cuda()
    lse = torch.logsumexp(x.double() @ w.double().t(), 1).float()
    g = (normal(4, rows) / rows).cuda()
    got, loss = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for call in (lambda: ops.linear_cross_entropy(x, w, targets, loss, got),
                 lambda: ops.linear_cross_entropy_backward(x, w, targets, lse, g, dx, dw)):
        call()
        with pytest.raises(FgError) as e:
            ops.sync()
        assert e.value.status == _lib.FG_ETIMEOUT
    _lib.check(ops.lib.ts_set_wait_limit(ops.h, 2_000_000_000, 0))
    x[(targets < 0) | (targets >= vocab)] = 0.0
    dx, dw = run_backward(ops, x, w, targets, lse, g, None, BF16, F32, 4, 0)
    check_backward(x, w, targets, lse, g, None, dx, dw)
