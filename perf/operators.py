"""Measured cases of the training-step operators: layer norm, 8-bit activation
checkpoints and their use in the backward pass, and token log probabilities.

`run` computes a case in plain float32 torch operations, or, when `own` is
true, through the package's TrainingOps.  A case's `op` names the operator:

  norm, norm_back           layer norm and its gradients
  checkpoint                activations to 8 bits and back
  act_back                  an activation's derivative from its saved output
  weight_grad               a matmul's weight gradient from its saved input
  logprobs, logprobs_back   token log probabilities and their gradient

A checkpoint is one byte buffer: rows of `pitch` int8 values (the columns
rounded up to 128), then rows of pitch / 32 scale bytes.  A block of 32
columns with scale byte E holds the values q * 2^(E - 133), or NaN for E = 255.
"""
import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the RNN language model chain's frame: a small batch, where latency counts
        {"name": "norm_64x1024_f32", "op": "norm", "rows": 64, "cols": 1024, "x": "f32", "y": "f32", "ckpt": False, "pad": 0},
        # a float32 residual stream normalised into a matmul's bf16 operand, checkpointed on the way
        {"name": "norm_8192x4096_ckpt", "op": "norm", "rows": 8192, "cols": 4096, "x": "f32", "y": "bf16", "ckpt": True, "pad": 0},
        # the gradient of a full batch in bf16
        {"name": "norm_back_8192x4096_bf16", "op": "norm_back", "rows": 8192, "cols": 4096, "x": "bf16", "y": "bf16", "ckpt": False, "pad": 0},
        # odd sizes, from the 8-bit checkpoint
        {"name": "norm_back_1021x5003_ckpt", "op": "norm_back", "rows": 1021, "cols": 5003, "x": "f32", "y": "f32", "ckpt": True, "pad": 0},
        # activations saved and brought back, full batch
        {"name": "checkpoint_8192x4096_f32", "op": "checkpoint", "rows": 8192, "cols": 4096, "x": "f32", "pad": 0},
        # the derivative of a tanh layer, ragged width inside a padded buffer
        {"name": "act_back_4097x4100_tanh", "op": "act_back", "rows": 4097, "cols": 4100, "x": "bf16", "act": "tanh", "pad": 28},
        # the sufficient factors' sizes: few tokens, a large weight
        {"name": "weight_grad_512x4096x4096", "op": "weight_grad", "rows": 512, "cols": 4096, "n": 4096, "affine": False, "pad": 0},
        # a full batch through a layer norm's affine input, with the bias gradient
        {"name": "weight_grad_8192x4096x4096", "op": "weight_grad", "rows": 8192, "cols": 4096, "n": 4096, "affine": True, "pad": 0},
        # scoring one step of a small batch of sequences
        {"name": "logprobs_16x32000_f32", "op": "logprobs", "rows": 16, "cols": 32000, "x": "f32", "k": 8, "pad": 0},
        # scoring a whole batch, odd vocabulary padded to a multiple of 64
        {"name": "logprobs_4096x50001_bf16", "op": "logprobs", "rows": 4096, "cols": 50001, "x": "bf16", "k": 20, "pad": 47},
        # the loss gradient with an entropy term
        {"name": "logprobs_back_2048x65536_f32", "op": "logprobs_back", "rows": 2048, "cols": 65536, "x": "f32", "entropy": True, "pad": 0},
        # a short ragged batch without the entropy term, rows that start at odd elements
        {"name": "logprobs_back_33x50001_bf16", "op": "logprobs_back", "rows": 33, "cols": 50001, "x": "bf16", "entropy": False, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "checkpoint", "act_back", "weight_grad", "logprobs", "logprobs_back"])
    pad = rng.choice([0, 0, 0, 1, 5, 8, 32, 77])
    x = rng.choice(["f32", "bf16"])
    if op == "weight_grad":
        n = _log_int(rng, 8, 4096)
        if rng.random() < 0.6:
            n = max(8, n // 8 * 8)
        return {"op": op, "rows": _log_int(rng, 1, 8192), "cols": _log_int(rng, 32, 4096), "n": n,
                "affine": rng.random() < 0.5, "pad": rng.choice([0, 0, 8, 3])}
    if op in ("logprobs", "logprobs_back"):
        cols = _log_int(rng, 100, 131072)
        rows = _log_int(rng, 1, max(1, min(4096, 2048 * 65536 // cols)))
        if op == "logprobs":
            return {"op": op, "rows": rows, "cols": cols, "x": x, "k": rng.choice([0, 1, 5, 8, 20, 32]), "pad": pad}
        return {"op": op, "rows": rows, "cols": cols, "x": x, "entropy": rng.random() < 0.5, "pad": pad}
    cols = _log_int(rng, 17, 16384)
    if rng.random() < 0.5:
        cols = max(32, cols // 32 * 32)
    rows = _log_int(rng, 1, max(1, min(65536, 8192 * 4096 // cols)))
    case = {"op": op, "rows": rows, "cols": cols, "x": x, "pad": pad}
    if op == "act_back":
        case["act"] = rng.choice(["relu", "sigmoid", "tanh"])
    elif op != "checkpoint":
        case["y"] = rng.choice(["f32", "bf16"])
        case["ckpt"] = rng.random() < 0.4
    return case


# ---- inputs ------------------------------------------------------------------


def _pitch(cols):
    return (cols + 127) // 128 * 128


def _step(e):
    """2^(e - 133) of scale bytes, NaN for 255."""
    e = e.to(torch.int32)
    return torch.where(e < 255, ((e - 6) << 23).view(torch.float32), float("nan"))


def _encode(x):
    """Values, columns in whole blocks of 32 -> int8 values and scale bytes."""
    blocks = x.unflatten(1, (-1, 32))
    top = blocks.abs().amax(2)
    e = (top.view(torch.int32) >> 23).clamp(min=7)
    q = (blocks / _step(e)[..., None]).nan_to_num(0.0).round().clamp(-127, 127)
    return q.to(torch.int8).flatten(1), e.to(torch.uint8)


def _decode(buf, rows, cols):
    """A checkpoint buffer's values in float32."""
    pitch = _pitch(cols)
    q = buf[:rows * pitch].view(torch.int8).view(rows, pitch // 32, 32).to(torch.float32)
    e = buf[rows * pitch:rows * pitch + rows * pitch // 32].view(rows, pitch // 32, 1)
    return (q * _step(e)).flatten(1)[:, :cols]


def _saved(x):
    """A float32 matrix as a checkpoint buffer."""
    rows, cols = x.shape
    q, e = _encode(torch.nn.functional.pad(x, (0, _pitch(cols) - cols)))
    return torch.cat([q.view(torch.uint8).flatten(), e.flatten()])


def _matrix(shape, dtype, pad, device="cuda"):
    """An uninitialised matrix whose rows lie `pad` elements further apart."""
    rows, cols = shape
    return torch.empty((rows, cols + pad), dtype=dtype, device=device)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, op, pad = case["rows"], case["cols"], case["op"], case["pad"]

    def normal(r, c, dtype, scale=1.0):
        out = _matrix((r, c), dtype, pad)
        return out.copy_(torch.randn((r, c), generator=gen, device="cuda") * scale)

    def vector(n, scale=1.0, shift=0.0):
        return torch.randn(n, generator=gen, device="cuda") * scale + shift

    s = {"case": case}
    if op in ("norm", "norm_back"):
        xt, yt = DTYPES[case["x"]], DTYPES[case["y"]]
        x = normal(rows, cols, xt, 1.5)
        x += 0.3
        s["gamma"], s["beta"] = vector(cols, 0.1, 1.0), vector(cols, 0.1)
        s["mean"], s["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        if op == "norm":
            s["x"], s["y"] = x, _matrix((rows, cols), yt, pad)
            if case["ckpt"]:
                s["buf"] = torch.empty(rows * _pitch(cols) // 32 * 33, dtype=torch.uint8, device="cuda")
                s["values"] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
            return s
        f = x.float()
        s["mean"] = f.mean(1)
        s["rstd"] = (f.var(1, unbiased=False) + EPS).rsqrt()
        s["dy"] = normal(rows, cols, yt)
        if case["ckpt"]:
            s["buf"] = _saved((f - s["mean"][:, None]) * s["rstd"][:, None])
        else:
            s["x"] = x
        s["dx"] = _matrix((rows, cols), xt, pad)
        s["dgamma"], s["dbeta"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    elif op == "checkpoint":
        s["x"] = normal(rows, cols, DTYPES[case["x"]])
        s["buf"] = torch.empty(rows * _pitch(cols) // 32 * 33, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    elif op == "act_back":
        act = {"relu": torch.relu, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[case["act"]]
        s["buf"] = _saved(act(torch.randn((rows, cols), generator=gen, device="cuda")))
        s["dy"] = normal(rows, cols, DTYPES[case["x"]])
        s["dx"] = _matrix((rows, cols), DTYPES[case["x"]], pad)
    elif op == "weight_grad":
        s["buf"] = _saved(torch.randn((rows, cols), generator=gen, device="cuda"))
        s["dy"] = normal(rows, case["n"], torch.bfloat16, 0.1)
        s["dw"] = torch.empty((cols, case["n"]), device="cuda")
        if case["affine"]:
            s["gamma"], s["beta"] = vector(cols, 0.1, 1.0), vector(cols, 0.1)
            s["db"] = torch.empty(case["n"], device="cuda")
    else:
        s["logits"] = normal(rows, cols, DTYPES[case["x"]], 2.5)
        s["tokens"] = torch.randint(0, cols, (rows,), generator=gen, device="cuda")
        if op == "logprobs":
            for name in ("logprob", "entropy", "lse"):
                s[name] = torch.empty(rows, device="cuda")
            k = min(case["k"], cols)
            if k:
                s["top_logprob"] = torch.empty((rows, k), device="cuda")
                s["top_id"] = torch.empty((rows, k), dtype=torch.int32, device="cuda")
        else:
            f = s["logits"].float()
            s["lse"] = torch.logsumexp(f, 1)
            s["entropy"] = s["lse"] - (torch.exp(f - s["lse"][:, None]) * f).sum(1)
            s["g_logprob"] = vector(rows, 0.1, -1.0)
            s["g_entropy"] = vector(rows, 0.01) if case["entropy"] else None
            s["dlogits"] = _matrix((rows, cols), DTYPES[case["x"]], pad)
    return s


# ---- one pass ------------------------------------------------------------------

_handle = None


def _own_run(s):
    global _handle
    from group_execution_gb300 import Checkpoint, TrainingOps
    if _handle is None:
        _handle = TrainingOps()
    ops, case = _handle, s["case"]
    op, rows, cols = case["op"], case["rows"], case["cols"]
    ckpt = Checkpoint(rows, cols, s["buf"]) if "buf" in s else None
    if op == "norm":
        ops.layer_norm(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], eps=EPS, ckpt=ckpt)
        out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        if ckpt:
            ops.checkpoint_load(ckpt, s["values"])
            out["values"] = s["values"]
        return out
    if op == "norm_back":
        ops.layer_norm_backward(s["dy"], ckpt or s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "checkpoint":
        ops.checkpoint_save(s["x"], ckpt)
        ops.checkpoint_load(ckpt, s["values"])
        return {"values": s["values"]}
    if op == "act_back":
        ops.activation_backward(case["act"], s["dy"], ckpt, s["dx"])
        return {"dx": s["dx"]}
    if op == "weight_grad":
        if not case["affine"]:
            ops.weight_grad(ckpt, s["dy"], s["dw"])
            return {"dw": s["dw"]}
        ops.weight_grad(ckpt, s["dy"], s["dw"], db=s["db"], gamma=s["gamma"], beta=s["beta"])
        return {"dw": s["dw"], "db": s["db"]}
    if op == "logprobs":
        ops.token_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["lse"], s.get("top_logprob"), s.get("top_id"))
        return {k: s[k] for k in ("logprob", "entropy", "lse", "top_logprob", "top_id") if k in s}
    ops.token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], s["g_logprob"], s["g_entropy"], s["dlogits"])
    return {"dlogits": s["dlogits"]}


def _plain_values(x):
    """What a checkpoint of float32 x stands for."""
    cols = x.shape[1]
    q, e = _encode(torch.nn.functional.pad(x, (0, -cols % 32)))
    return (q.to(torch.float32).unflatten(1, (-1, 32)) * _step(e)[..., None]).flatten(1)[:, :cols].to(torch.bfloat16)


def _plain_run(s):
    case = s["case"]
    op, rows, cols = case["op"], case["rows"], case["cols"]
    if op == "norm":
        x = s["x"].float()
        mean = x.sum(1) / cols
        d = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).sum(1) / cols + EPS)
        h = d * rstd[:, None]
        out = {"y": (h * s["gamma"] + s["beta"]).to(DTYPES[case["y"]]), "mean": mean, "rstd": rstd}
        if case["ckpt"]:
            out["values"] = _plain_values(h)
        return out
    if op == "norm_back":
        h = _decode(s["buf"], rows, cols) if case["ckpt"] else (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        a = dy * s["gamma"]
        c1, c2 = a.sum(1) / cols, (a * h).sum(1) / cols
        dx = s["rstd"][:, None] * (a - c1[:, None] - h * c2[:, None])
        return {"dx": dx.to(DTYPES[case["x"]]), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}
    if op == "checkpoint":
        return {"values": _plain_values(s["x"].float())}
    if op == "act_back":
        a, dy = _decode(s["buf"], rows, cols), s["dy"].float()
        slope = {"relu": lambda: (a > 0).float(), "sigmoid": lambda: a * (1 - a), "tanh": lambda: 1 - a * a}[case["act"]]()
        return {"dx": (dy * slope).to(DTYPES[case["x"]])}
    if op == "weight_grad":
        x, dy = _decode(s["buf"], rows, cols), s["dy"].float()
        if not case["affine"]:
            return {"dw": x.t() @ dy}
        return {"dw": (x * s["gamma"] + s["beta"]).t() @ dy, "db": dy.sum(0)}
    x, at = s["logits"].float(), s["tokens"][:, None]
    if op == "logprobs":
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - top)
        total = e.sum(1)
        lse = top[:, 0] + torch.log(total)
        out = {"logprob": x.gather(1, at)[:, 0] - lse, "entropy": torch.log(total) - (e * (x - top)).sum(1) / total, "lse": lse}
        k = min(case["k"], cols)
        if k:
            del e
            value, index = torch.sort(x, dim=1, descending=True, stable=True)
            out["top_logprob"] = value[:, :k] - lse[:, None]
            out["top_id"] = index[:, :k].to(torch.int32)
        return out
    logp = x - s["lse"][:, None]
    p = torch.exp(logp)
    dx = p * -s["g_logprob"][:, None]
    if s["g_entropy"] is not None:
        dx -= s["g_entropy"][:, None] * p * (logp + s["entropy"][:, None])
    dx.scatter_add_(1, at, s["g_logprob"][:, None])
    return {"dlogits": dx.to(DTYPES[case["x"]])}


def run(state):
    return _own_run(state) if own else _plain_run(state)


# ---- the definitions in 64 bits ------------------------------------------------


def _exact_values(buf, rows, cols):
    pitch = (cols + 127) & ~127
    raw = buf.to(torch.int64)
    q = raw[:rows * pitch].reshape(rows, pitch)[:, :cols]
    q = torch.where(q > 127, q - 256, q).double()
    e = raw[rows * pitch:].reshape(rows, pitch // 32).repeat_interleave(32, dim=1)[:, :cols].double()
    return q * torch.exp2(e - 133.0)


def _exact_rounded(x):
    """x in 64 bits at its checkpoint's precision, in blocks of 32 of a row."""
    rows, cols = x.shape
    b = torch.cat([x, x.new_zeros(rows, -cols % 32)], 1).reshape(-1, 32)
    top = torch.linalg.vector_norm(b, float("inf"), dim=1, keepdim=True).clamp(min=2.0 ** -126)
    step = torch.exp2(torch.frexp(top).exponent.double() - 7.0).clamp(min=2.0 ** -126)
    return (torch.round(b / step).clamp(-127, 127) * step).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op, rows, cols = case["op"], case["rows"], case["cols"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        h = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
        out = {"y": h * s["gamma"].double() + s["beta"].double(), "mean": mean, "rstd": rstd}
        if case["ckpt"]:
            out["values"] = _exact_rounded(h)
        return out
    if op == "norm_back":
        rstd = s["rstd"].double().unsqueeze(1)
        if case["ckpt"]:
            h = _exact_values(s["buf"], rows, cols)
        else:
            h = (s["x"].double() - s["mean"].double().unsqueeze(1)) * rstd
        dy = s["dy"].double()
        g = dy * s["gamma"].double()
        dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        return {"dx": dx, "dgamma": torch.einsum("ij,ij->j", dy, h), "dbeta": dy.sum(0)}
    if op == "checkpoint":
        return {"values": _exact_rounded(s["x"].double())}
    if op == "act_back":
        a = _exact_values(s["buf"], rows, cols)
        slope = torch.sign(a).clamp(min=0) if case["act"] == "relu" else a - a ** 2 if case["act"] == "sigmoid" else 1 - a ** 2
        return {"dx": slope * s["dy"].double()}
    if op == "weight_grad":
        x, dy = _exact_values(s["buf"], rows, cols), s["dy"].double()
        if not case["affine"]:
            return {"dw": torch.mm(x.T, dy)}
        return {"dw": torch.mm((x * s["gamma"].double() + s["beta"].double()).T, dy), "db": dy.sum(0)}
    x = s["logits"].double()
    logp = torch.log_softmax(x, 1)
    if op == "logprobs":
        out = {"logprob": logp[torch.arange(rows, device="cuda"), s["tokens"]], "entropy": -(logp.exp() * logp).sum(1),
               "lse": torch.logsumexp(x, 1)}
        k = min(case["k"], cols)
        if k:
            ids = torch.argsort(-x, dim=1, stable=True)[:, :k]
            out["top_logprob"], out["top_id"] = logp.gather(1, ids), ids.to(torch.int32)
        return out
    # the gradient takes lse and entropy as they were saved, in 32 bits
    logp = x - s["lse"].double().unsqueeze(1)
    g = torch.zeros_like(x)
    g[torch.arange(rows, device="cuda"), s["tokens"]] = 1.0
    g = s["g_logprob"].double().unsqueeze(1) * (g - logp.exp())
    if case["entropy"]:
        g -= s["g_entropy"].double().unsqueeze(1) * logp.exp() * (logp + s["entropy"].double().unsqueeze(1))
    return {"dlogits": g}


def work(case):
    rows, cols, op = case["rows"], case["cols"], case["op"]
    size = {"f32": 4, "bf16": 2}
    cells = rows * cols
    saved = rows * ((cols + 31) // 32) * 33
    if op == "norm":
        moved = cells * (size[case["x"]] + size[case["y"]]) + 8 * cols + 8 * rows
        if case["ckpt"]:
            moved += 2 * saved + 2 * cells
        return {"bytes": moved, "flops": 8 * cells}
    if op == "norm_back":
        read = saved if case["ckpt"] else cells * size[case["x"]]
        return {"bytes": read + cells * (size[case["x"]] + size[case["y"]]) + 12 * cols + 8 * rows, "flops": 14 * cells}
    if op == "checkpoint":
        return {"bytes": cells * (size[case["x"]] + 2) + 2 * saved, "flops": 4 * cells}
    if op == "act_back":
        return {"bytes": saved + 2 * cells * size[case["x"]], "flops": 4 * cells}
    if op == "weight_grad":
        n = case["n"]
        return {"bytes": saved + 2 * rows * n + 4 * cols * n, "flops": 2 * cells * n}
    if op == "logprobs":
        return {"bytes": cells * size[case["x"]] + rows * (20 + 8 * case["k"]), "flops": 6 * cells}
    return {"bytes": 2 * cells * size[case["x"]] + 24 * rows, "flops": 6 * cells}
