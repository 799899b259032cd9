"""Training-step operators in float64: layer norm, 8-bit checkpoints and the
gradients that read them, token log probabilities."""
import numpy as np


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd, normalised rows)."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    h = d * rstd[:, None]
    y = h * (1.0 if gamma is None else np.asarray(gamma, np.float64))
    return y + (0.0 if beta is None else np.asarray(beta, np.float64)), mean, rstd, h


def layer_norm_backward(dy, h, rstd, gamma=None):
    """(dx, dgamma, dbeta) from the normalised rows h."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    u = dy * (1.0 if gamma is None else np.asarray(gamma, np.float64))
    c1, c2 = u.mean(1, keepdims=True), (u * h).mean(1, keepdims=True)
    return np.asarray(rstd, np.float64)[:, None] * (u - c1 - h * c2), (dy * h).sum(0), dy.sum(0)


def pitch(cols):
    return (cols + 127) // 128 * 128


def checkpoint_encode(x):
    """The checkpoint buffer's bytes of a float32 matrix."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    p = pitch(cols)
    b = np.zeros((rows, p), np.float32)
    b[:, :cols] = x
    b = b.reshape(rows, p // 32, 32)
    finite = np.isfinite(b).all(2)
    top = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0)).max(2), 1.0).astype(np.float64)
    _, ex = np.frexp(top)                       # top = m 2^ex with m in [0.5, 1)
    e = np.where(top > 0, np.maximum(ex + 126, 7), 7)
    e = np.where(finite, e, 255)
    step = np.ldexp(1.0, np.where(finite, e, 133) - 133)
    q = np.where(finite[..., None], np.rint(np.where(finite[..., None], b, 0).astype(np.float64) / step[..., None]), 0)
    q = np.clip(q, -127, 127).astype(np.int8)
    return np.concatenate([q.reshape(-1).view(np.uint8), e.astype(np.uint8).reshape(-1)])


def checkpoint_decode(buf, rows, cols):
    p = pitch(cols)
    q = buf[:rows * p].view(np.int8).reshape(rows, p // 32, 32).astype(np.float64)
    e = buf[rows * p:rows * p + rows * p // 32].reshape(rows, p // 32).astype(np.int64)
    step = np.where(e < 255, np.ldexp(1.0, np.minimum(e, 254) - 133), np.nan)
    return (q * step[..., None]).reshape(rows, p)[:, :cols]


def checkpoint_steps(buf, rows, cols):
    """Every value's step."""
    p = pitch(cols)
    e = buf[rows * p:rows * p + rows * p // 32].reshape(rows, p // 32).astype(np.int64)
    return np.repeat(np.ldexp(1.0, e - 133), 32, axis=1)[:, :cols]


def activation_backward(op, dy, a):
    """dy f'(x) from a = f(x)."""
    slope = {"relu": lambda: np.where(np.isnan(a), a, a > 0), "sigmoid": lambda: a * (1 - a), "tanh": lambda: 1 - a * a}[op]()
    return np.asarray(dy, np.float64) * slope


def weight_grad(h, dy, gamma=None, beta=None):
    """(dw, db): X^T dy with X = gamma h + beta by column, and dy's column sums."""
    x = np.asarray(h, np.float64)
    if gamma is not None:
        x = x * np.asarray(gamma, np.float64)
    if beta is not None:
        x = x + np.asarray(beta, np.float64)
    dy = np.asarray(dy, np.float64)
    return x.T @ dy, dy.sum(0)


def token_logprobs(x, tokens, k=0):
    """(logprob, entropy, lse, top_logprob, top_id).  -inf logits have
    probability 0; a row of nothing else has lse -inf and entropy 0; a token
    outside the vocabulary leaves its row's logprob 0."""
    x = np.asarray(x, np.float64)
    rows, vocab = x.shape
    with np.errstate(all="ignore"):
        top = np.where(np.isnan(x).any(1), np.nan, x.max(1))
        none = top == -np.inf
        base = np.where(none, 0.0, top)
        d = x - base[:, None]
        e = np.exp(d)
        s = e.sum(1)
        lse = np.where(none, -np.inf, base + np.log(s))
        ent = np.where(none, 0.0, np.log(s) - np.where(e == 0, 0.0, e * d).sum(1) / s)
    lp = np.zeros(rows)
    for r, t in enumerate(tokens):
        if 0 <= t < vocab:
            lp[r] = -np.inf if none[r] else x[r, t] - lse[r]
    order = np.argsort(-np.where(np.isnan(x), np.inf, x), axis=1, kind="stable") if not np.isnan(x).any() else \
        np.stack([np.lexsort((np.arange(vocab), np.where(np.isnan(r), 0, -r), ~np.isnan(r))) for r in x])
    ids = order[:, :k].astype(np.int32)
    with np.errstate(invalid="ignore"):
        tlp = np.where(none[:, None], -np.inf, np.take_along_axis(x, ids.astype(np.int64), 1) - lse[:, None])
    return lp, ent, lse, tlp, ids


def token_logprobs_backward(x, tokens, g_logprob, g_entropy=None):
    """dlogits from the gradients of logprob and entropy."""
    x = np.asarray(x, np.float64)
    rows, vocab = x.shape
    _, ent, lse, _, _ = token_logprobs(x, tokens)
    out = np.zeros_like(x)
    for r in range(rows):
        if lse[r] == -np.inf:
            continue
        lp = x[r] - lse[r]
        p = np.exp(lp)
        t = int(tokens[r])
        if 0 <= t < vocab:
            out[r] = -g_logprob[r] * p
            out[r, t] += g_logprob[r]
        if g_entropy is not None:
            out[r] -= g_entropy[r] * np.where(p == 0, 0.0, p * (np.where(p == 0, 0.0, lp) + ent[r]))
    return out
