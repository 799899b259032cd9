"""One training step of a small language model's last layers, built from the
package's pieces: layer norm, two matmul groups with their tails, token log
probabilities, the gradients of all of them, and the packing of the gradients
for the exchange.

What the backward pass needs of the activations is kept in 8 bits: the
normalised rows (for the first weight's gradient and the layer norm's) and the
relu's output (for its derivative and the second weight's gradient).

    python examples/training_step.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from group_execution_gb300 import Checkpoint, Graph, TensorFusion, TrainingOps  # noqa: E402


def _matmul(rows, inner, cols, trans_b=False, bias_relu=False):
    """A plan of one matmul group, bf16 x bf16 -> f32 [rows, cols], with an
    optional bias and relu tail, and a function that launches it."""
    g = Graph()
    a = g.input((rows, inner), "bf16")
    b = g.input((cols, inner) if trans_b else (inner, cols), "bf16")
    bias = g.input((cols,)) if bias_relu else None
    out = g.op("matmul_bf16", (a, b), (0, int(trans_b)))
    if bias_relu:
        out = g.op("relu", (g.op("badd_col", (out, bias)),))
    g.mark_output(out)
    plan = g.build()
    assert plan.n_groups == 1

    def launch(x, w, y, b1=None):
        plan.launch_group(0, {a: x, b: w, out: y} | ({bias: b1} if bias_relu else {}))

    return launch


class Model:
    """norm -> matmul, bias, relu -> matmul -> log probabilities."""

    def __init__(self, tokens=512, width=256, hidden=1024, vocab=4000, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=gen, device="cuda") * scale

        self.tokens, self.width, self.hidden, self.vocab = tokens, width, hidden, vocab
        self.gamma, self.beta = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
        self.w1, self.b1 = normal(width, hidden, scale=width ** -0.5), torch.zeros(hidden, device="cuda")
        self.w2 = normal(hidden, vocab, scale=hidden ** -0.5)
        self.params = [self.gamma, self.beta, self.w1, self.b1, self.w2]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.ops = TrainingOps()
        self.fusion = TensorFusion(self.grads)
        self.packed = torch.empty(self.fusion.total_bytes, dtype=torch.uint8, device="cuda")
        # activations: bf16 operands of the matmuls, the 8-bit checkpoints
        f32 = dict(dtype=torch.float32, device="cuda")
        b16 = dict(dtype=torch.bfloat16, device="cuda")
        self.normed, self.acts = torch.empty((tokens, width), **b16), torch.empty((tokens, hidden), **b16)
        self.saved_norm, self.saved_acts = Checkpoint(tokens, width), Checkpoint(tokens, hidden)
        self.relu, self.logits = torch.empty((tokens, hidden), **f32), torch.empty((tokens, vocab), **f32)
        self.mean, self.rstd = torch.empty(tokens, **f32), torch.empty(tokens, **f32)
        self.logprob, self.entropy, self.lse = (torch.empty(tokens, **f32) for _ in range(3))
        self.dlogits, self.dhidden = torch.empty((tokens, vocab), **b16), torch.empty((tokens, hidden), **b16)
        self.dacts, self.dnormed = torch.empty((tokens, hidden), **f32), torch.empty((tokens, width), **f32)
        self.dx = torch.empty((tokens, width), **f32)
        self.up = _matmul(tokens, width, hidden, bias_relu=True)
        self.out = _matmul(tokens, hidden, vocab)
        self.out_back = _matmul(tokens, vocab, hidden, trans_b=True)
        self.up_back = _matmul(tokens, hidden, width, trans_b=True)

    def step(self, x, targets):
        """Forward and backward: the gradients (float32 and packed), the loss."""
        ops = self.ops
        w1, w2 = self.w1.bfloat16(), self.w2.bfloat16()
        # forward
        ops.layer_norm(x, self.gamma, self.beta, self.normed, self.mean, self.rstd, ckpt=self.saved_norm)
        self.up(self.normed, w1, self.relu, self.b1)
        ops.checkpoint_save(self.relu, self.saved_acts)
        ops.checkpoint_load(self.saved_acts, self.acts)
        self.out(self.acts, w2, self.logits)
        ops.token_logprobs(self.logits, targets, self.logprob, self.entropy, self.lse)
        # backward of the mean negative log probability
        g = torch.full((self.tokens,), -1.0 / self.tokens, device="cuda")
        dgamma, dbeta, dw1, db1, dw2 = self.grads
        ops.token_logprobs_backward(self.logits, targets, self.lse, None, g, None, self.dlogits)
        ops.weight_grad(self.saved_acts, self.dlogits, dw2)
        self.out_back(self.dlogits, w2, self.dacts)
        ops.activation_backward("relu", self.dacts, self.saved_acts, self.dhidden)
        ops.weight_grad(self.saved_norm, self.dhidden, dw1, db=db1, gamma=self.gamma, beta=self.beta)
        self.up_back(self.dhidden, w1, self.dnormed)
        ops.layer_norm_backward(self.dnormed, self.saved_norm, self.gamma, None, self.rstd, self.dx, dgamma, dbeta)
        self.fusion.pack(1.0, self.packed)
        return -self.logprob.mean()


def main(steps=20, rate=0.5):
    model = Model()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((model.tokens, model.width), generator=gen, device="cuda")
    targets = torch.randint(0, model.vocab, (model.tokens,), generator=gen, device="cuda")
    losses = []
    for _ in range(steps):
        losses.append(model.step(x, targets))
        model.fusion.unpack(1.0, model.packed)   # what came back from the exchange
        for p, d in zip(model.params, model.grads):
            p -= rate * d
    model.ops.sync()
    return [float(v) for v in losses]


if __name__ == "__main__":
    for i, loss in enumerate(main(*(int(a) for a in sys.argv[1:2]))):
        print(f"step {i}: loss {loss:.4f}")
