"""Train a small recurrent language model with the library's operators, then run it token by token.

    python -m gated_delta_rule_12_gb300.train_example --steps 60

One training step goes through everything the library has for it: layer norm, the gated delta rule
(``chunk_fwd`` / ``chunk_bwd``), the per-channel gated scan, and the linear softmax cross entropy, whose gradient
starts the way back.  The linear projections between them are plain matrix products, which are the model's own.
Afterwards the trained model reads a sequence one token at a time with ``decode_step`` and ``gated_scan_step``; its
hidden states have to agree with those of the parallel pass.

The task: predict the token seen ``--lag`` positions ago.  With a fixed seed the loss starts at log(vocab) and falls.
"""
import argparse
import math

import torch

import gated_delta_rule_12_gb300 as gdn

HEADS, DIM = 2, 128          # of the gated delta rule
D = HEADS * DIM


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = gdn.layer_norm_fwd(x, weight, bias)
        ctx.save_for_backward(x, mean, rstd, weight)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        return gdn.layer_norm_bwd(dy.contiguous(), x, mean, rstd, weight)


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        out, _ = gdn.chunk_fwd(q, k, v, g, beta, output_final_state=False)
        ctx.save_for_backward(q, k, v, g, beta)
        return out

    @staticmethod
    def backward(ctx, dout):
        return gdn.chunk_bwd(*ctx.saved_tensors, dout.contiguous(), want_dinit=False)[:5]


class GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g):
        out, _ = gdn.gated_scan_fwd(x, g, input_gate=True, output_final_state=False)
        ctx.save_for_backward(x, g, out)
        return out

    @staticmethod
    def backward(ctx, dout):
        return gdn.gated_scan_bwd(*ctx.saved_tensors, dout.contiguous(), input_gate=True, want_dinit=False)[:2]


class LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, weight, targets):
        loss, lse = gdn.linear_cross_entropy_fwd(h, weight, targets)
        ctx.save_for_backward(h, weight, targets, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        return (*gdn.linear_cross_entropy_bwd(*ctx.saved_tensors, dloss.contiguous()), None)


class Model(torch.nn.Module):
    """Two residual layers, a gated delta rule and a gated scan, each behind a layer norm; fp32 parameters, bf16
    activations."""

    def __init__(self, vocab):
        super().__init__()
        self.embed = torch.nn.Parameter(0.5 * torch.randn(vocab, D))
        self.head = torch.nn.Parameter(D ** -0.5 * torch.randn(vocab, D))
        self.norms = torch.nn.ParameterList([p for _ in range(3) for p in (torch.ones(D), torch.zeros(D))])
        # q, k, v; the gates of the rule; the scan's input and gate; the two ways back into the residual stream
        self.proj = torch.nn.ParameterList([D ** -0.5 * torch.randn(D, n) for n in (3 * D, 2 * HEADS, 2 * D)] +
                                           [0.5 * D ** -0.5 * torch.randn(D, D) for _ in range(2)])

    def delta_inputs(self, y):
        q, k, v = (y @ self.proj[0].bfloat16()).view(*y.shape[:-1], 3, HEADS, DIM).unbind(-3)
        a, b = (y.float() @ self.proj[1]).view(*y.shape[:-1], 2, HEADS).unbind(-2)
        g = -0.1 * torch.nn.functional.softplus(a)
        return q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), torch.sigmoid(b).contiguous()

    def scan_inputs(self, y):
        x, z = (y @ self.proj[2].bfloat16()).view(*y.shape[:-1], 2, D).unbind(-2)
        return x.contiguous(), torch.nn.functional.logsigmoid(z.float() + 1).bfloat16().contiguous()

    def forward(self, tokens):
        """[B, T] tokens to [B, T, D] hidden states in front of the head."""
        x = self.embed[tokens].bfloat16()
        y = LayerNorm.apply(x, self.norms[0], self.norms[1])
        x = x + DeltaRule.apply(*self.delta_inputs(y)).flatten(-2) @ self.proj[3].bfloat16()
        y = LayerNorm.apply(x, self.norms[2], self.norms[3])
        x = x + GatedScan.apply(*self.scan_inputs(y)) @ self.proj[4].bfloat16()
        return LayerNorm.apply(x, self.norms[4], self.norms[5])

    def loss(self, tokens, targets):
        """The mean loss over the targets that are not ignored (negative)."""
        h = self(tokens).view(-1, D)
        return LinearCrossEntropy.apply(h, self.head.bfloat16(), targets.view(-1)).sum() / (targets >= 0).sum()

    @torch.no_grad()
    def step(self, token, states):
        """One token per sequence [B] to [B, D], the two recurrent states moving on in place."""
        x = self.embed[token].bfloat16()
        y = gdn.layer_norm_fwd(x, self.norms[0], self.norms[1])[0]
        x = x + gdn.decode_step(states[0], *self.delta_inputs(y)).flatten(-2) @ self.proj[3].bfloat16()
        y = gdn.layer_norm_fwd(x, self.norms[2], self.norms[3])[0]
        x = x + gdn.gated_scan_step(states[1], *self.scan_inputs(y), input_gate=True) @ self.proj[4].bfloat16()
        return gdn.layer_norm_fwd(x, self.norms[4], self.norms[5])[0]

    def states(self, B):
        dev = self.embed.device
        return [torch.zeros(B, HEADS, DIM, DIM, device=dev), torch.zeros(B, D, device=dev)]


def train(steps=60, batch=8, length=256, vocab=512, lag=2, seed=0, report=print):
    """Returns the losses and the relative difference of the token-by-token pass from the parallel one."""
    gdn.load_library()
    torch.manual_seed(seed)
    model = Model(vocab).cuda()
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    losses = []
    for i in range(steps):
        tokens = torch.randint(0, vocab, (batch, length), generator=gen, device="cuda")
        targets = torch.full_like(tokens, -100)          # the first positions have nothing to recall
        targets[:, lag:] = tokens[:, :-lag]
        opt.zero_grad()
        loss = model.loss(tokens, targets.int())
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if i % 10 == 0 or i == steps - 1:
            report(f"step {i}: loss {losses[-1]:.3f} (log vocab {math.log(vocab):.3f})")
    with torch.no_grad():
        tokens = tokens[:, :64]
        parallel, states = model(tokens).float(), model.states(batch)
        serial = torch.stack([model.step(tokens[:, t].contiguous(), states) for t in range(tokens.shape[1])], 1).float()
    off = ((serial - parallel).norm() / parallel.norm()).item()
    report(f"token by token against the parallel pass: relative difference {off:.2e}")
    return losses, off


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 60), ("batch", 8), ("length", 256), ("vocab", 512), ("lag", 2), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    if not torch.cuda.is_available():
        raise SystemExit("train_example needs a CUDA device")
    train(a.steps, a.batch, a.length, a.vocab, a.lag, a.seed)


if __name__ == "__main__":
    main()
