"""The token operators together, as a small language model's last layers use them.

    python examples/next_token.py [--steps 8] [--batch 4]

Serving: a batch of hidden states goes through the final norm, which hands out 8-bit
tokens, through the 8-bit output head, and a token of each row is drawn; the token's
embedding is mixed into the state for the next step.  Training: the norm's gain and bias
are fitted to given outputs with the gradients of the backward pass.

Weights are random: the program shows the calls, not a model.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_dequant_dot_gb300 as loom  # noqa: E402


class Head:
    """Final norm, 8-bit output head and sampling for `width` features and `vocab` tokens."""

    def __init__(self, width: int, vocab: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.width = vocab, width
        self.embedding = torch.randn(vocab, width, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
        weight = torch.randn(vocab, width, generator=g, device="cuda") * width ** -0.5
        # the head's rows as bytes, laid out once: the tokens' own quantisation serves for rows of weights
        self.weight, self.scale = loom.loom_quantize_tokens(weight)
        self.gain, self.bias = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")

    def logits(self, x):
        q, scale = loom.loom_layer_norm_i8(x, self.gain, self.bias)
        return loom.loom_i8_matmul(self.weight, self.scale, self.vocab, self.width, q, scale, x.shape[0], y_dtype=torch.bfloat16)[0]

    def next_token(self, x, uniform, **settings):
        return loom.loom_sample_tokens(self.logits(x), uniform, **settings)

    def generate(self, x, steps: int, seed: int = 1, **settings):
        """(tokens [steps][batch], log probabilities) from hidden states x [batch][width]."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        tokens, logprobs = [], []
        for _ in range(steps):
            token, logprob = self.next_token(x, torch.rand(x.shape[0], generator=g, device="cuda"), **settings)
            x = (0.5 * x.float() + self.embedding[token.long()].float()).to(x.dtype)
            tokens.append(token)
            logprobs.append(logprob)
        return torch.stack(tokens), torch.stack(logprobs)


def fit_norm(x, target, steps: int = 60, rate: float = 0.5):
    """Gain and bias of a layer norm of x fitted to `target` by gradient descent; the losses."""
    rows, width = x.shape
    gain, bias = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
    losses = []
    for _ in range(steps):
        y, mean, rstd = loom.loom_layer_norm(x, gain, bias)
        error = y.float() - target.float()
        losses.append(float(error.square().mean()))
        dy = (error * (2.0 / rows)).to(x.dtype)
        _, dgain, dbias = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, want_dx=False)
        gain -= rate * dgain
        bias -= rate * dbias
    return gain, bias, losses


def main():
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--steps", type=int, default=8)
    a.add_argument("--batch", type=int, default=4)
    a.add_argument("--width", type=int, default=1024)
    a.add_argument("--vocab", type=int, default=16384)
    args = a.parse_args()
    head = Head(args.width, args.vocab)
    x = torch.randn(args.batch, args.width, device="cuda").to(torch.bfloat16)
    tokens, logprobs = head.generate(x, args.steps, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
    for b in range(args.batch):
        print("row %d: tokens %s, log probability %.3f" % (b, tokens[:, b].tolist(), float(logprobs[:, b].sum())))
    rows = torch.randn(512, args.width, device="cuda")
    want_gain, want_bias = 1 + 0.3 * torch.randn(args.width, device="cuda"), torch.randn(args.width, device="cuda")
    target = loom.loom_layer_norm(rows, want_gain, want_bias, want_stats=False)[0]
    gain, bias, losses = fit_norm(rows, target)
    print("norm fitted: loss %.4f -> %.2g, gain off by %.2g at most" % (losses[0], losses[-1], float((gain - want_gain).abs().max())))


if __name__ == "__main__":
    main()
