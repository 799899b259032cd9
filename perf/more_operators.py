"""Measured cases of the vocabulary's two ends of a training step: the embedding
of tokens and its gradient, and the softmax cross entropy of a linear layer over
the vocabulary with its gradients.

`run` computes a case in plain float32 torch operations, or, when `own` is
true, through the package's TrainingOps.  A case's `op` names the operator:

  embed, embed_back     rows of a table by token, scaled; the table's gradient
  loss, loss_back       cross entropy of x w^T without its logits; dx and dw

The table and the weight w are [vocab, cols], a row a token.  A token or a
target of -1 marks a padded place: it embeds to zeros, and is not scored.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one step of a small batch of sequences: a lookup where latency counts
        {"name": "embed_16x1024_f32", "op": "embed", "rows": 16, "cols": 1024, "vocab": 32000, "table": "f32", "y": "f32", "pad": 0, "none": 0.0},
        # a full batch from a bf16 table into a float32 residual stream
        {"name": "embed_8192x4096_bf16", "op": "embed", "rows": 8192, "cols": 4096, "vocab": 50001, "table": "bf16", "y": "f32", "pad": 0, "none": 0.1},
        # the example's step: few tokens, a small table, its whole gradient
        {"name": "embed_back_512x256_f32", "op": "embed_back", "rows": 512, "cols": 256, "vocab": 4000, "dy": "f32", "table": "f32", "accumulate": False, "pad": 0, "none": 0.0},
        # a full batch in bf16 into a float32 gradient that is written whole
        {"name": "embed_back_8192x4096_bf16", "op": "embed_back", "rows": 8192, "cols": 4096, "vocab": 50001, "dy": "bf16", "table": "f32", "accumulate": False, "pad": 0, "none": 0.1},
        # tied weights: added to what the loss left there; many tokens, odd width
        {"name": "embed_back_65536x1003_tied", "op": "embed_back", "rows": 65536, "cols": 1003, "vocab": 50001, "dy": "f32", "table": "f32", "accumulate": True, "pad": 5, "none": 0.05},
        # scoring one step of a small batch: the weight is read once
        {"name": "loss_16x1024x32000", "op": "loss", "rows": 16, "cols": 1024, "vocab": 32000, "pad": 0, "none": 0.0},
        # a batch of a narrow model over an odd vocabulary
        {"name": "loss_4096x1024x50001", "op": "loss", "rows": 4096, "cols": 1024, "vocab": 50001, "pad": 0, "none": 0.1},
        # a full batch of a wide model
        {"name": "loss_8192x4096x50001", "op": "loss", "rows": 8192, "cols": 4096, "vocab": 50001, "pad": 0, "none": 0.1},
        # the example's step
        {"name": "loss_back_512x1024x4000", "op": "loss_back", "rows": 512, "cols": 1024, "vocab": 4000, "lse": False, "pad": 0, "none": 0.0},
        # a ragged batch, odd width in a padded buffer, with a gradient of lse
        {"name": "loss_back_1021x1003x50001", "op": "loss_back", "rows": 1021, "cols": 1003, "vocab": 50001, "lse": True, "pad": 5, "none": 0.3},
        # the batch of a narrow model
        {"name": "loss_back_4096x1024x50001", "op": "loss_back", "rows": 4096, "cols": 1024, "vocab": 50001, "lse": False, "pad": 0, "none": 0.1},
        # a full batch of a wide model
        {"name": "loss_back_8192x4096x50001", "op": "loss_back", "rows": 8192, "cols": 4096, "vocab": 50001, "lse": False, "pad": 0, "none": 0.1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["embed", "embed_back", "loss", "loss_back"])
    case = {"op": op, "none": rng.choice([0.0, 0.0, 0.1, 0.6])}
    if op in ("loss", "loss_back"):
        rows, cols, vocab = _log_int(rng, 1, 16384), _log_int(rng, 64, 4096), _log_int(rng, 100, 131072)
        if rng.random() < 0.7:
            cols = max(64, cols // 64 * 64)
        rows = max(1, min(rows, 8192 * 4096 * 50001 // (cols * vocab)))
        case |= {"rows": rows, "cols": cols, "vocab": vocab}
        # rows on 16 bytes, or (one in six) wherever the width puts them
        case["pad"] = rng.choice([-cols % 8] * 4 + [-cols % 8 + 8, 0])
        if op == "loss_back":
            case["lse"] = rng.random() < 0.4
        return case
    cols = _log_int(rng, 33, 8192)
    if rng.random() < 0.6:
        cols = max(64, cols // 64 * 64)
    case |= {"cols": cols, "vocab": _log_int(rng, 100, min(131072, 50001 * 4096 // cols)),
             "rows": _log_int(rng, 1, min(65536, 65536 * 1003 // cols)), "pad": rng.choice([0, 0, 0, 1, 5, 8]),
             "table": rng.choice(["f32", "bf16"])}
    if op == "embed":
        case["y"] = rng.choice(["f32", "bf16"])
    else:
        case["dy"], case["accumulate"] = rng.choice(["f32", "bf16"]), rng.random() < 0.5
    return case


# ---- inputs ------------------------------------------------------------------


def _matrix(shape, dtype, pad):
    """An uninitialised matrix whose rows lie `pad` elements further apart."""
    rows, cols = shape
    return torch.empty((rows, cols + pad), dtype=dtype, device="cuda")[:, :cols]


def _scale(case):
    return float(case["cols"]) ** 0.5


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, vocab, op, pad = case["rows"], case["cols"], case["vocab"], case["op"], case["pad"]

    def normal(r, c, dtype, scale=1.0):
        return _matrix((r, c), dtype, pad).copy_(torch.randn((r, c), generator=gen, device="cuda") * scale)

    # token frequencies of text: the r-th most frequent one as 1 / r, the ranks
    # spread over the vocabulary
    rank = torch.exp(torch.rand(rows, generator=gen, device="cuda", dtype=torch.float64) * torch.log(torch.tensor(vocab + 1.0))) - 1
    ids = torch.randperm(vocab, generator=gen, device="cuda")[rank.long().clamp(0, vocab - 1)]
    ids[torch.rand(rows, generator=gen, device="cuda") < case["none"]] = -1
    s = {"case": case, "ids": ids}
    if op == "embed":
        s["table"] = normal(vocab, cols, DTYPES[case["table"]], cols ** -0.5)
        s["y"] = _matrix((rows, cols), DTYPES[case["y"]], pad)
    elif op == "embed_back":
        s["dy"] = normal(rows, cols, DTYPES[case["dy"]])
        s["dtable"] = _matrix((vocab, cols), DTYPES[case["table"]], pad)
        if case["accumulate"]:   # what the loss left in the gradient; every pass adds to it
            s["dtable"] = normal(vocab, cols, DTYPES[case["table"]])
    else:
        s["x"], s["w"] = normal(rows, cols, torch.bfloat16), normal(vocab, cols, torch.bfloat16, 2.5 * cols ** -0.5)
        if op == "loss":
            s["loss"], s["lse"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            return s
        # what the forward pass saved
        s["lse"] = torch.cat([torch.logsumexp(x @ s["w"].float().t(), 1) for x in s["x"].float().split(4096)])
        scored = (ids >= 0).sum().clamp(min=1)
        s["g_loss"] = (torch.rand(rows, generator=gen, device="cuda") + 0.5) / scored
        s["g_lse"] = torch.randn(rows, generator=gen, device="cuda") * 0.01 / scored if case["lse"] else None
        s["dx"], s["dw"] = _matrix((rows, cols), torch.bfloat16, pad), _matrix((vocab, cols), torch.bfloat16, pad)
    return s


# ---- one pass ------------------------------------------------------------------

_handle = None


def _own_run(s):
    global _handle
    from group_execution_gb300 import TrainingOps
    if _handle is None:
        _handle = TrainingOps(workspace_bytes=1 << 30)
    ops, case = _handle, s["case"]
    op = case["op"]
    if op == "embed":
        ops.embedding(s["ids"], s["table"], s["y"], scale=_scale(case))
        return {"y": s["y"]}
    if op == "embed_back":
        ops.embedding_backward(s["ids"], s["dy"], s["dtable"], scale=_scale(case), accumulate=case["accumulate"])
        return {"dtable": s["dtable"]}
    if op == "loss":
        ops.linear_cross_entropy(s["x"], s["w"], s["ids"], s["loss"], s["lse"])
        return {"loss": s["loss"], "lse": s["lse"]}
    ops.linear_cross_entropy_backward(s["x"], s["w"], s["ids"], s["lse"], s["g_loss"], s["dx"], s["dw"], g_lse=s["g_lse"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _plain_run(s):
    case, ids = s["case"], s["ids"]
    op = case["op"]
    there = ids >= 0
    at = ids.clamp(min=0)
    if op == "embed":
        return {"y": (s["table"][at].float() * _scale(case) * there[:, None]).to(DTYPES[case["y"]])}
    if op == "embed_back":
        out = torch.zeros((case["vocab"], case["cols"]), device="cuda")
        out.index_add_(0, at, s["dy"].float() * (there[:, None] * _scale(case)))
        if case["accumulate"]:
            out += s["dtable"]
        s["dtable"].copy_(out)
        return {"dtable": s["dtable"]}
    x, w = s["x"].float(), s["w"].float()
    logits = x @ w.t()
    if op == "loss":
        top = logits.amax(1)
        lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
        return {"loss": torch.where(there, lse - logits.gather(1, at[:, None])[:, 0], 0.0), "lse": lse}
    g = s["g_loss"] * there
    logits -= s["lse"][:, None]
    d = torch.exp(logits, out=logits)
    d *= (g if s["g_lse"] is None else g + s["g_lse"])[:, None]
    d.scatter_add_(1, at[:, None], -g[:, None])
    return {"dx": (d @ w).to(torch.bfloat16), "dw": (d.t() @ x).to(torch.bfloat16)}


def run(state):
    return _own_run(state) if own else _plain_run(state)


# ---- the definitions in 64 bits ------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op, rows, cols, vocab, ids = case["op"], case["rows"], case["cols"], case["vocab"], s["ids"]
    used = torch.nonzero(ids >= 0)[:, 0]
    if op == "embed":
        y = torch.zeros((rows, cols), dtype=torch.float64, device="cuda")
        y[used] = s["table"].double()[ids[used]] * _scale(case)
        return {"y": y}
    if op == "embed_back":
        # the tokens that stand together in sorted order, by differences of
        # running sums taken column block by column block
        order = used[torch.argsort(ids[used])]
        keys, count = torch.unique_consecutive(ids[order], return_counts=True)
        out = torch.zeros((vocab, cols), dtype=torch.float64, device="cuda")
        if case["accumulate"]:
            out += s["dtable"]
        ends = torch.cumsum(count, 0)
        for c in range(0, cols, 512):
            run_sum = torch.cumsum(s["dy"][:, c:c + 512].double()[order], 0)
            run_sum = torch.cat([run_sum.new_zeros((1, run_sum.shape[1])), run_sum])
            out[keys, c:c + 512] += _scale(case) * (run_sum[ends] - run_sum[ends - count])
        return {"dtable": out}
    x, w = s["x"].double(), s["w"].double()
    if op == "loss":
        lse, loss = [], []
        for k in range(0, rows, 2048):
            logits = torch.einsum("tc,vc->tv", x[k:k + 2048], w)
            i = ids[k:k + 2048]
            lse.append(torch.logsumexp(logits, 1))
            nll = torch.nn.functional.cross_entropy(logits, i, ignore_index=-1, reduction="none")
            loss.append(nll)
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    # the gradient takes lse as it was saved, in 32 bits
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for k in range(0, rows, 2048):
        r = slice(k, min(rows, k + 2048))
        p = torch.exp(torch.mm(x[r], w.T) - s["lse"][r].double().unsqueeze(1))
        g = torch.where(ids[r] >= 0, s["g_loss"][r].double(), 0.0)
        h = 0.0 if s["g_lse"] is None else s["g_lse"][r].double()
        p *= (g + h).unsqueeze(1)
        here = torch.nonzero(ids[r] >= 0)[:, 0]
        p[here, ids[r][here]] -= g[here]
        dx[r] = torch.mm(p, w)
        dw += torch.mm(p.T, x[r])
    return {"dx": dx, "dw": dw}


def work(case):
    rows, cols, vocab, op = case["rows"], case["cols"], case["vocab"], case["op"]
    size = {"f32": 4, "bf16": 2}
    used = rows * (1 - case["none"])
    if op == "embed":
        return {"bytes": used * cols * size[case["table"]] + rows * cols * size[case["y"]] + 8 * rows, "flops": rows * cols}
    if op == "embed_back":
        # the gradient is written whole, or the rows in use are read and written
        # (of `used` tokens about this many are different ones)
        different = min(vocab, used / (1 + used / vocab) ** 0.5)
        out = (2 * different if case["accumulate"] else vocab) * cols * size[case["table"]]
        return {"bytes": used * cols * size[case["dy"]] + out + 8 * rows, "flops": 2 * used * cols}
    both = (rows + vocab) * cols * 2
    if op == "loss":
        return {"bytes": both + 16 * rows, "flops": 2 * rows * cols * vocab}
    return {"bytes": 2 * both + 20 * rows, "flops": 6 * rows * cols * vocab}
