"""A training step of one residual block that keeps its activations in 8 bits, on the library's operators.

A feed-forward block between two norms, with a gate per sequence:

    h  = norm(r) g_in                                            sf_sandwich_norm_forward (r kept in 8 bits)
    a  = relu(h Wup^T),  x = a Wdown^T                           sf_gemm_abt_bf16; a kept: sf_checkpoint_store
    s  = r + scale gate norm(x) g_post,  h' = norm(s) g_pre      sf_sandwich_norm_forward (x and s kept)

and backwards, from the three checkpoints and four vectors of norms alone:

    dr, dx, dg_post, dg_pre, dgate                               sf_sandwich_norm_backward
    dWdown = dx^T a;  da = dx Wdown                              sf_checkpoint_wgrad; sf_gemm_bf16
    h again from r's checkpoint, dWup = da^T h, dh = da Wup      sf_checkpoint_load; sf_gemm_bf16
    dr, dg_in                                                    sf_sandwich_norm_backward
    AdamW on the weights, gains and gates                        sf_adamw_layer_step

    python examples/residual_block.py [--sequences B] [--tokens N] [--hidden D] [--ffn F] [--steps K]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from layer_optimizer_gb300 import native  # noqa: E402

BF = torch.bfloat16


class ResidualBlock:
    """bf16 weights, fp32 masters and moments, all buffers allocated once; `sequences` of `tokens` rows each."""

    def __init__(self, sequences, tokens, hidden, ffn, scale=0.5, eps=1e-5, group=128, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rows = sequences * tokens
        self.rows, self.hidden, self.ffn, self.group, self.device = rows, hidden, ffn, group, device
        normal = lambda *shape: 0.02 * torch.randn(*shape, generator=g, device=device)  # noqa: E731
        self.masters = dict(up=normal(ffn, hidden), down=normal(hidden, ffn), gate=1.0 + normal(sequences, hidden),
                            g_in=torch.ones(hidden, device=device), g_post=torch.ones(hidden, device=device),
                            g_pre=torch.ones(hidden, device=device))
        self.weights = {k: m.to(BF) for k, m in self.masters.items()}
        self.grads = {k: torch.empty_like(w) for k, w in self.weights.items()}
        self.moments = {k: (torch.zeros_like(m), torch.zeros_like(m)) for k, m in self.masters.items()}
        self.layer = [native.make_tensor(self.grads[k], m, *self.moments[k], self.weights[k]) for k, m in self.masters.items()]
        self.entry = native.sandwich(eps)
        self.end = native.sandwich(eps, block_scale=scale, gate_span=tokens)
        self.r8, self.x8, self.s8 = (self._kept(hidden) for _ in range(3))
        self.a8 = self._kept(ffn)
        self.rstd_in, self.rstd_post, self.rstd_pre = (torch.empty(rows, device=device) for _ in range(3))
        self.norm_ws = self._scratch(native.sf_sandwich_norm_workspace_bytes(rows, hidden))
        self.down_ws = self._scratch(native.sf_checkpoint_wgrad_workspace_bytes(rows, hidden, ffn))
        self.step_no = 0

    def _kept(self, cols):
        n = -(-cols // self.group) if self.group else 1
        return native.checkpoint(torch.empty(self.rows, cols, dtype=torch.float8_e4m3fn, device=self.device),
                                 torch.empty(self.rows, n, dtype=torch.float8_e8m0fnu, device=self.device), self.group)

    def _scratch(self, size):
        return torch.empty(max(16, size), dtype=torch.uint8, device=self.device)

    def _bf(self, *shape):
        return torch.empty(*shape, dtype=BF, device=self.device)

    def _product(self, A, a_layout, B, b_layout, M, N, K):
        C = torch.empty(M, N, device=self.device)
        native.sf_gemm_bf16(A, a_layout, B, b_layout, C, M, N, K, A.stride(0), B.stride(0), N)
        return C.to(BF)

    def forward(self, r):
        """s and h of the next block; what the backward pass needs stays in the checkpoints."""
        w, n, d, f = self.weights, self.rows, self.hidden, self.ffn
        h, s, h_next = self._bf(n, d), self._bf(n, d), self._bf(n, d)
        native.sf_sandwich_norm_forward(self.entry, r, gain_pre=w["g_in"], h=h, sum8=self.r8, rstd_pre=self.rstd_in)
        a = torch.relu_(self._product(h, 0, w["up"], 0, n, f, d))
        native.sf_checkpoint_store(a, self.a8)
        x = self._product(a, 0, w["down"], 0, n, d, f)
        native.sf_sandwich_norm_forward(self.end, x, r, gain_post=w["g_post"], gain_pre=w["g_pre"], gate=w["gate"], sum=s, h=h_next,
                                        x8=self.x8, sum8=self.s8, rstd_post=self.rstd_post, rstd_pre=self.rstd_pre)
        return s, h_next

    def backward(self, dh_next, ds):
        """The gradient of r, and the weights' into self.grads, from the gradients of h_next and s."""
        w, g, n, d, f = self.weights, self.grads, self.rows, self.hidden, self.ffn
        dr, dx = self._bf(n, d), self._bf(n, d)
        native.sf_sandwich_norm_backward(self.end, dh=dh_next, dsum=ds, x=self.x8, sum=self.s8, gain_post=w["g_post"],
                                         gain_pre=w["g_pre"], gate=w["gate"], rstd_post=self.rstd_post, rstd_pre=self.rstd_pre,
                                         dresidual=dr, dx=dx, dgain_post=g["g_post"], dgain_pre=g["g_pre"], dgate=g["gate"],
                                         ws=self.norm_ws)
        native.sf_checkpoint_wgrad(dx, self.a8, g["down"], ws=self.down_ws)
        da = self._product(dx, 0, w["down"], 1, n, f, d)
        a, h = self._bf(n, f), self._bf(n, d)
        native.sf_checkpoint_load(self.a8, a)
        da.masked_fill_(a == 0, 0.0)
        native.sf_checkpoint_load(self.r8, h, row_factor=self.rstd_in, gain=w["g_in"])
        g["up"].copy_(self._product(da, 1, h, 1, f, d, n))
        dh = self._product(da, 0, w["up"], 1, n, d, f)
        out = self._bf(n, d)
        native.sf_sandwich_norm_backward(self.entry, dh=dh, dsum=dr, sum=self.r8, gain_pre=w["g_in"], rstd_pre=self.rstd_in, dx=out,
                                         dgain_pre=g["g_in"], ws=self.norm_ws)
        return out

    def update(self, hp):
        self.step_no += 1
        native.sf_adamw_layer_step(self.layer, hp, self.step_no)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=11008)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = a.sequences * a.tokens
    draw = lambda: torch.randn(rows, a.hidden, generator=g, device="cuda").to(BF)  # noqa: E731
    r, dh, ds = draw(), 1e-3 * draw(), 1e-3 * draw()
    block, hp = ResidualBlock(a.sequences, a.tokens, a.hidden, a.ffn), native.hparams(lr=1e-4)

    def step():
        block.forward(r)
        block.backward(dh, ds)
        block.update(hp)

    step()
    native.sf_sync_status()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        step()
    end.record()
    end.synchronize()
    kept = sum(c.values.rows * c.values.cols for c in (block.r8, block.x8, block.s8, block.a8))
    print(f"{start.elapsed_time(end) / a.steps:.3f} ms a step ({rows} tokens, hidden {a.hidden}, feed-forward {a.ffn}); "
          f"{kept / 2 ** 20:.0f} MiB of activations kept (in bf16 {kept / 2 ** 19:.0f})")


if __name__ == "__main__":
    main()
