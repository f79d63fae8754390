"""Trains a Markov drafting head on a synthetic language, then drafts with it.

One training step is the path that include/dspark_head.h declares:

    r    = residual + dropout(x)                  dspark_residual_norm
    h    = r / rms(r) * gain
    loss = cross entropy of h W^T + U[prev] V^T   dspark_head_loss
    gradients of h, W, U, V                       dspark_head_loss_grad
    gradients of gain, x, residual                dspark_residual_norm_grad

followed by plain gradient descent with momentum on fp32 copies of the factors.
The language: the next token is one of two fixed functions of the previous one,
into the lower or the upper half of the vocabulary, and the row's residual
stream says which: h W^T has to learn the half, U V^T the functions.  The head
then drafts greedily with dspark_chain_lmhead, from the same bf16 factors,
and the drafts are compared with the language.

    python examples/train_head.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_draft_dspark_gb300 import dspark as D  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import head as H  # noqa: E402

VOCAB, WIDTH, RANK = 256, 128, 64
ROWS, POSITIONS = 2048, 7
EPS, DROP = 1e-6, 0.1


class Language:
    """next = step[mode][token], in half `mode` of the vocabulary; the residual
    stream carries the mode."""

    def __init__(self, device, seed=0):
        g = torch.Generator().manual_seed(seed)
        half = VOCAB // 2
        self.step = torch.stack([m * half + torch.randint(0, half, (VOCAB,), generator=g)
                                 for m in range(2)]).to(device)
        self.sign = torch.randn(2, WIDTH, generator=g).to(device)
        self.g = torch.Generator(device=device).manual_seed(seed)
        self.device = device

    def rows(self, n):
        mode = torch.randint(0, 2, (n,), generator=self.g, device=self.device)
        prev = torch.randint(0, VOCAB, (n,), generator=self.g, device=self.device)
        noise = torch.randn(n, WIDTH, generator=self.g, device=self.device)
        residual = (self.sign[mode] + 0.3 * noise).bfloat16()
        x = (0.3 * torch.randn(n, WIDTH, generator=self.g, device=self.device)).bfloat16()
        target = self.step[mode, prev]
        # a tenth of the rows has no target (a prompt's, say)
        skip = torch.rand(n, generator=self.g, device=self.device) < 0.1
        return mode, x, residual, prev.int(), torch.where(skip, -1, target).int()


class Head:
    """fp32 factors and their bf16 copies, with one workspace for each call."""

    def __init__(self, device):
        g = torch.Generator(device=device).manual_seed(1)
        new = lambda sd, *s: torch.randn(*s, generator=g, device=device) * sd  # noqa: E731
        self.master = {"W": new(0.02, VOCAB, WIDTH), "U": new(0.1, VOCAB, RANK), "V": new(0.1, VOCAB, RANK),
                       "gain": torch.ones(WIDTH, device=device)}
        self.speed = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.p = {k: v.bfloat16() for k, v in self.master.items()}
        self.grad = {k: torch.empty_like(v) for k, v in self.p.items()}
        new16 = lambda: torch.empty(ROWS, WIDTH, dtype=torch.bfloat16, device=device)  # noqa: E731
        new32 = lambda: torch.empty(ROWS, device=device)  # noqa: E731
        self.r, self.h, self.dh, self.dx, self.dres = (new16() for _ in range(5))
        self.rstd, self.loss, self.lse = new32(), new32(), new32()
        self.head_ws = H.new_workspace(H.dspark_head_workspace_size(ROWS, VOCAB, WIDTH, RANK, True), device)
        self.norm_ws = H.new_workspace(H.dspark_norm_workspace_size(ROWS, WIDTH), device)

    def gradients(self, x, residual, prev, target, seed, offset):
        """Mean loss of the rows with a target; gradients in self.grad, those
        of x and residual in self.dx and self.dres."""
        p, g = self.p, self.grad
        drop = dict(p=DROP, seed=seed, offset=offset)
        dloss = (target >= 0).float()
        dloss /= dloss.sum().clamp(min=1.0)
        H.dspark_residual_norm(x, residual, p["gain"], self.r, self.h, None, self.rstd, eps=EPS, **drop)
        H.dspark_head_loss(self.h, p["W"], p["U"], p["V"], prev, target, self.loss, self.lse, self.head_ws)
        H.dspark_head_loss_grad(self.h, p["W"], p["U"], p["V"], prev, target, self.lse, dloss,
                                self.dh, g["W"], g["U"], g["V"], self.head_ws)
        H.dspark_residual_norm_grad(self.dh, None, self.r, p["gain"], self.rstd, self.dx, self.dres,
                                    g["gain"], self.norm_ws, **drop)
        return (self.loss * dloss).sum()

    def step(self, rate):
        for k, m in self.master.items():
            self.speed[k].mul_(0.9).add_(self.grad[k].float())
            m.sub_(self.speed[k], alpha=rate)
            self.p[k].copy_(m)


def draft(head, residual, last, positions):
    """Greedy drafts [N, positions] after the tokens `last`, all positions from
    the same residual stream, without dropout."""
    n = last.numel()
    h = torch.empty_like(residual)
    H.dspark_residual_norm(residual, None, head.p["gain"], None, h, eps=EPS)
    h = h[:, None, :].expand(n, positions, WIDTH).contiguous()
    out = torch.empty(n, positions, dtype=torch.int32, device=last.device)
    ws = D.new_workspace(D.dspark_chain_workspace_size(n, positions), last.device)
    D.dspark_chain_lmhead(h, head.p["W"], head.p["U"], head.p["V"], last, out, None, ws)
    assert D.dspark_read_status(ws) == 0
    return out


def main(steps=300, rate=2.0):
    device = torch.device("cuda:0")
    torch.cuda.set_device(device)
    language, head = Language(device), Head(device)
    losses = []
    for i in range(steps):
        _, x, residual, prev, target = language.rows(ROWS)
        loss = head.gradients(x, residual, prev, target, seed=7, offset=i)
        head.step(rate)
        if i % 50 == 0 or i == steps - 1:
            losses.append(loss.item())
            print(f"step {i:4d}  loss {losses[-1]:.4f}")
    mode, _, residual, prev, _ = language.rows(256)
    got = draft(head, residual, prev, POSITIONS)
    want, token = [], prev.long()
    for _ in range(POSITIONS):
        token = language.step[mode, token]
        want.append(token)
    right = (got == torch.stack(want, 1)).float().mean().item()
    print(f"{100 * right:.1f} % of {got.numel()} drafted tokens are the language's")
    return losses, right


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 300)
