"""A training step of a model's output end, with its update, on the library's operators.

The last block of a decoder hands over its output x and the residual stream r.
One step runs, all on the device:

    s, h, rstd = add_rmsnorm(r + dropout(x))          sf_add_rmsnorm_forward
    loss, dh, dW = cross_entropy(h W^T, labels)       lce_vocab_forward_backward
    dr, dx, dgain = gradients of the first line       sf_add_rmsnorm_backward
    AdamW on gain and W                               sf_adamw_layer_step

dr and dx are what the blocks below take.  The dropout mask is drawn again in
the backward pass from the step's offset, so nothing of it is kept; the
cross-entropy keeps no logits; dgain and dW come in bf16, as the update wants
them.  `checkpoint=True` writes h in 8 bits with scales beside it as well, for a copy of
the activations that crosses the host link in half the bytes; `restored()` is
how such a copy is read back.

    python examples/output_head.py [--tokens N] [--hidden D] [--vocab V] [--steps K]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from layer_optimizer_gb300 import native  # noqa: E402


class OutputHead:
    """Final norm and output layer: bf16 weights, fp32 masters and moments, all buffers allocated once."""

    def __init__(self, tokens, hidden, vocab, p=0.1, eps=1e-5, seed=0, device="cuda", checkpoint=False):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        bf = dict(dtype=torch.bfloat16, device=device)
        self.tokens, self.hidden, self.vocab, self.p, self.eps, self.seed = tokens, hidden, vocab, p, eps, seed
        self.masters = [torch.ones(hidden, device=device),
                        0.02 * torch.randn(vocab, hidden, generator=g, device=device)]
        self.weights = [m.to(torch.bfloat16) for m in self.masters]            # gain, W
        self.moments = [(torch.zeros_like(m), torch.zeros_like(m)) for m in self.masters]
        self.grads = [torch.empty_like(w) for w in self.weights]
        self.layer = [native.make_tensor(dw, m, e, v, w)
                      for dw, m, (e, v), w in zip(self.grads, self.masters, self.moments, self.weights)]
        self.s, self.h, self.dh = (torch.empty(tokens, hidden, **bf) for _ in range(3))
        self.dr, self.dx = (torch.empty(tokens, hidden, **bf) for _ in range(2))
        self.rstd, self.token_loss = torch.empty(tokens, device=device), torch.empty(tokens, device=device)
        self.loss = torch.empty(1, device=device)
        self.h8 = self.h8_scale = None
        if checkpoint:
            self.h8 = torch.empty(tokens, hidden, dtype=torch.float8_e4m3fn, device=device)
            self.h8_scale = torch.empty(tokens, -(-hidden // 128), device=device)
        self.norm_ws = torch.empty(native.sf_add_rmsnorm_workspace_bytes(tokens, hidden), dtype=torch.uint8, device=device)
        self.lce_ws = torch.empty(native.lce_vocab_workspace_bytes(tokens, hidden, vocab), dtype=torch.uint8, device=device)
        self.step_no = 0

    def forward_backward(self, x, r, labels, offset, train=True, stream=None):
        """Loss and gradients; `offset` names the step's dropout mask."""
        gain, W = self.weights
        p = self.p if train else 0.0
        rng = native.rng(self.seed, offset)
        native.sf_add_rmsnorm_forward(x, r, gain, self.eps, sum=self.s, h=self.h, h8=self.h8, h8_scale=self.h8_scale,
                                      group=128 if self.h8 is not None else 0, rstd=self.rstd, p=p, rng=rng, stream=stream)
        native.lce_vocab_forward_backward(self.h, W, labels, loss=self.loss, token_loss=self.token_loss, dH=self.dh,
                                          dW=self.grads[1], ws=self.lce_ws, stream=stream)
        native.sf_add_rmsnorm_backward(self.dh, self.s, gain, self.rstd, dresidual=self.dr, dx=self.dx,
                                       dgain=self.grads[0], p=p, rng=rng, ws=self.norm_ws, stream=stream)
        return self.loss

    def restored(self):
        """h in fp32 from its 8-bit copy: the stored values times their groups' scales."""
        return self.h8.float() * self.h8_scale.repeat_interleave(128, dim=1)[:, :self.hidden]

    def step(self, x, r, labels, hp, stream=None):
        """One training step; returns the loss (on the device) and leaves dr, dx for the blocks below."""
        self.step_no += 1
        self.forward_backward(x, r, labels, self.step_no, stream=stream)
        native.sf_adamw_layer_step(self.layer, hp, self.step_no, stream=stream)
        return self.loss


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    draw = lambda: torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, r = draw(), draw()
    labels = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda", dtype=torch.int32)
    labels[: a.tokens // 4] = -100                                   # a prompt: no loss on its tokens
    head = OutputHead(a.tokens, a.hidden, a.vocab)
    hp = native.hparams(lr=1e-3)
    for k in range(a.steps):
        print(f"step {k + 1}: loss {head.step(x, r, labels, hp).item():.4f}")
    native.sf_sync_status()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        head.step(x, r, labels, hp)
    end.record()
    end.synchronize()
    print(f"{start.elapsed_time(end) / a.steps:.3f} ms a step ({a.tokens} tokens, hidden {a.hidden}, vocabulary {a.vocab})")


if __name__ == "__main__":
    main()
