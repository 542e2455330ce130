"""Train a small recurrent language model with the library's operators, then run it token by token.

    python -m gated_delta_rule_12_gb300.train_example --steps 60

One training step goes through what the library has for it: a norm, the gated delta rule
(``chunk_fwd`` / ``chunk_bwd``), the per-channel gated scan, and the linear softmax cross entropy, whose gradient
starts the way back.  The linear projections between them are plain matrix products, which are the model's own.
Afterwards the trained model reads a sequence one token at a time with ``decode_step`` and ``gated_scan_step``; its
hidden states have to agree with those of the parallel pass.

``--norm rms`` takes the root-mean-square norm with the residual's addition in place of layer norm, ``--entropy C`` trains
on the log probabilities with C times the distribution's entropy added, ``--score`` reports log probabilities, entropy and
alternatives of the last batch, and ``--fp8`` (with ``--norm rms``) runs the token-by-token pass once more with the
projections in 8 bits, from the norm's 8-bit output or a quantised one.

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


class RmsNorm(torch.autograd.Function):
    """The norm of x + residual, and that sum (without a residual: x)."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        y, s, rstd = gdn.rms_norm_fwd(x, weight, residual=residual)
        ctx.save_for_backward(x if s is None else s, rstd, weight)
        ctx.added = s is not None
        ctx.set_materialize_grads(False)
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, rstd, weight = ctx.saved_tensors
        dy = torch.zeros_like(s) if dy is None else dy.contiguous()
        dx, dw = gdn.rms_norm_bwd(dy, s, rstd, weight, dresidual=None if ds is None else ds.contiguous())
        return dx, dx if ctx.added else None, dw


class LinearLogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, weight, targets):
        logp, entropy, lse, _, _ = gdn.linear_log_probs_fwd(h, weight, targets)
        ctx.save_for_backward(h, weight, targets, lse, entropy)
        return logp, entropy

    @staticmethod
    def backward(ctx, dlogp, dentropy):
        return (*gdn.linear_log_probs_bwd(*ctx.saved_tensors, dlogp.contiguous(), dentropy.contiguous()), None)


class Model(torch.nn.Module):
    """Two residual layers, a gated delta rule and a gated scan, each behind a norm; fp32 parameters, bf16 activations."""

    def __init__(self, vocab, norm="layer"):
        super().__init__()
        self.rms = norm == "rms"
        self.embed = torch.nn.Parameter(0.5 * torch.randn(vocab, D))
        self.head = torch.nn.Parameter(D ** -0.5 * torch.randn(vocab, D))
        one = (torch.ones, torch.zeros)[:1 if self.rms else 2]   # the norm's weight, and the layer norm's bias
        self.norms = torch.nn.ParameterList([make(D) for _ in range(3) for make in one])
        # q, k, v; the gates of the rule; the scan's input and gate; the two ways back into the residual stream
        self.proj = torch.nn.ParameterList([D ** -0.5 * torch.randn(D, n) for n in (3 * D, 2 * HEADS, 2 * D)] +
                                           [0.5 * D ** -0.5 * torch.randn(D, D) for _ in range(2)])

    def project(self, i, y):
        return y.float() @ self.proj[1] if i == 1 else y @ self.proj[i].bfloat16()

    def delta_inputs(self, y, project=None):
        project = project or self.project
        q, k, v = (t for t in project(0, y).unflatten(-1, (3, HEADS, DIM)).unbind(-3))
        a, b = project(1, y).unflatten(-1, (2, HEADS)).unbind(-2)
        g = -0.1 * torch.nn.functional.softplus(a)
        return q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), torch.sigmoid(b).contiguous()

    def scan_inputs(self, y, project=None):
        x, z = (project or self.project)(2, y).unflatten(-1, (2, D)).unbind(-2)
        return x.contiguous(), torch.nn.functional.logsigmoid(z.float() + 1).bfloat16().contiguous()

    def forward(self, tokens):
        """[B, T] tokens to [B, T, D] hidden states in front of the head."""
        x = self.embed[tokens].bfloat16()
        if self.rms:
            y, _ = RmsNorm.apply(x, None, self.norms[0])
            y, x = RmsNorm.apply(DeltaRule.apply(*self.delta_inputs(y)).flatten(-2) @ self.proj[3].bfloat16(), x,
                                 self.norms[1])
            return RmsNorm.apply(GatedScan.apply(*self.scan_inputs(y)) @ self.proj[4].bfloat16(), x, self.norms[2])[0]
        y = LayerNorm.apply(x, self.norms[0], self.norms[1])
        x = x + DeltaRule.apply(*self.delta_inputs(y)).flatten(-2) @ self.proj[3].bfloat16()
        y = LayerNorm.apply(x, self.norms[2], self.norms[3])
        x = x + GatedScan.apply(*self.scan_inputs(y)) @ self.proj[4].bfloat16()
        return LayerNorm.apply(x, self.norms[4], self.norms[5])

    def loss(self, tokens, targets, entropy=0.0):
        """The mean loss over the targets that are not ignored (negative), less ``entropy`` times the mean entropy."""
        h, head, t = self(tokens).view(-1, D), self.head.bfloat16(), targets.view(-1)
        if entropy:
            logp, H = LinearLogProbs.apply(h, head, t)
            return -(logp + entropy * H).sum() / (targets >= 0).sum()
        return LinearCrossEntropy.apply(h, head, t).sum() / (targets >= 0).sum()

    @torch.no_grad()
    def step(self, token, states):
        """One token per sequence [B] to [B, D], the two recurrent states moving on in place."""
        x = self.embed[token].bfloat16()
        if self.rms:
            y = gdn.rms_norm_fwd(x, self.norms[0])[0]
            o = gdn.decode_step(states[0], *self.delta_inputs(y)).flatten(-2) @ self.proj[3].bfloat16()
            y, x, _ = gdn.rms_norm_fwd(o, self.norms[1], residual=x)
            o = gdn.gated_scan_step(states[1], *self.scan_inputs(y), input_gate=True) @ self.proj[4].bfloat16()
            return gdn.rms_norm_fwd(o, self.norms[2], residual=x)[0]
        y = gdn.layer_norm_fwd(x, self.norms[0], self.norms[1])[0]
        x = x + gdn.decode_step(states[0], *self.delta_inputs(y)).flatten(-2) @ self.proj[3].bfloat16()
        y = gdn.layer_norm_fwd(x, self.norms[2], self.norms[3])[0]
        x = x + gdn.gated_scan_step(states[1], *self.scan_inputs(y), input_gate=True) @ self.proj[4].bfloat16()
        return gdn.layer_norm_fwd(x, self.norms[4], self.norms[5])[0]

    @torch.no_grad()
    def quantize(self):
        """The projections' weights in 8 bits."""
        return [gdn.fp8_quantize(p.t().contiguous(), block_rows=128) for p in self.proj]

    @torch.no_grad()
    def step_fp8(self, token, states, weights):
        """``step`` with the projections in 8 bits, ``weights`` from ``quantize``."""
        def project(i, y):
            out = gdn.fp8_linear(*y, *weights[i])
            return out.float() if i == 1 else out

        x = self.embed[token].bfloat16()
        y = gdn.rms_norm_fp8(x, self.norms[0])[:2]
        o = gdn.decode_step(states[0], *self.delta_inputs(y, project)).flatten(-2)
        *y, x = gdn.rms_norm_fp8(project(3, gdn.fp8_quantize(o)), self.norms[1], residual=x)
        o = gdn.gated_scan_step(states[1], *self.scan_inputs(y, project), input_gate=True)
        return gdn.rms_norm_fwd(project(4, gdn.fp8_quantize(o)), self.norms[2], residual=x)[0]

    def states(self, B):
        dev = self.embed.device
        return [torch.zeros(B, HEADS, DIM, DIM, device=dev), torch.zeros(B, D, device=dev)]


def train(steps=60, batch=8, length=256, vocab=512, lag=2, seed=0, report=print, norm="layer", entropy=0.0, score=False,
          fp8=False):
    """Returns the losses and the relative difference of the token-by-token pass from the parallel one; with ``fp8`` that of
    the pass with 8-bit projections too."""
    if fp8 and norm != "rms":
        raise ValueError("the 8-bit pass takes the root-mean-square norm: norm='rms'")
    gdn.load_library()
    torch.manual_seed(seed)
    model = Model(vocab, norm).cuda()
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    losses = []
    for i in range(steps):
        tokens = torch.randint(0, vocab, (batch, length), generator=gen, device="cuda")
        targets = torch.full_like(tokens, -100)          # the first positions have nothing to recall
        targets[:, lag:] = tokens[:, :-lag]
        opt.zero_grad()
        loss = model.loss(tokens, targets.int(), entropy)
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if i % 10 == 0 or i == steps - 1:
            report(f"step {i}: loss {losses[-1]:.3f} (log vocab {math.log(vocab):.3f})")
    with torch.no_grad():
        full, tokens = tokens, tokens[:, :64]
        parallel, states = model(tokens).float(), model.states(batch)
        serial = torch.stack([model.step(tokens[:, t].contiguous(), states) for t in range(tokens.shape[1])], 1).float()
        if score:
            t = targets.int().view(-1)
            logp, H, _, ids, _ = gdn.linear_log_probs_fwd(model(full).view(-1, D), model.head.bfloat16(), t, top_k=5)
            kept = (t >= 0).sum().item()
            report(f"last batch: mean log probability {logp.sum().item() / kept:.3f}, entropy {H.sum().item() / kept:.3f}, "
                   f"{((ids == t[:, None]) & (t >= 0)[:, None]).any(-1).sum().item() / kept:.0%} among the best 5")
        if fp8:
            weights, states = model.quantize(), model.states(batch)
            in8 = torch.stack([model.step_fp8(tokens[:, t].contiguous(), states, weights) for t in range(tokens.shape[1])], 1)
    off = ((serial - parallel).norm() / parallel.norm()).item()
    report(f"token by token against the parallel pass: relative difference {off:.2e}")
    if not fp8:
        return losses, off
    off8 = ((in8.float() - parallel).norm() / parallel.norm()).item()
    report(f"the same with projections in 8 bits: relative difference {off8:.2e}")
    return losses, off, off8


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 60), ("batch", 8), ("length", 256), ("vocab", 512), ("lag", 2), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--norm", choices=["layer", "rms"], default="layer")
    ap.add_argument("--entropy", type=float, default=0.0, help="weight of the entropy in the objective")
    ap.add_argument("--score", action="store_true", help="report log probabilities and alternatives of the last batch")
    ap.add_argument("--fp8", action="store_true", help="token by token with 8-bit projections too (with --norm rms)")
    a = ap.parse_args(argv)
    if not torch.cuda.is_available():
        raise SystemExit("train_example needs a CUDA device")
    if a.fp8 and a.norm != "rms":
        ap.error("--fp8 takes --norm rms")
    train(a.steps, a.batch, a.length, a.vocab, a.lag, a.seed, norm=a.norm, entropy=a.entropy, score=a.score, fp8=a.fp8)


if __name__ == "__main__":
    main()
