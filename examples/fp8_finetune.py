"""A fine-tuning step and a rollout with 8-bit projections: the FP8 operators and the cross entropy as they are used.

A small residual network whose projections run in FP8 (``fp8_linear``: forward, input gradient and weight gradient; the
activation and the addition to the FP32 residual stream are in the products' epilogues) below a BF16 vocabulary head
whose loss is ``linear_cross_entropy`` (with a little label smoothing and z-loss, no logits kept) is trained on a
synthetic task: the next token is a fixed permutation of the present one.  Then the head is quantised once, in 128 x 128
blocks, and the trained network's tokens are scored twice, as a rollout with an 8-bit head and a BF16 trainer would: FP8
logits of single tokens through ``logp_fwd``, and the fused BF16 head.  The difference of the two log-probabilities is
the drift that an importance ratio between them sees.

    python examples/fp8_finetune.py [--steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vocab_selected_token_tile_gb300 as rlk  # noqa: E402
from vocab_selected_token_tile_gb300.autograd import fp8_linear, linear_cross_entropy  # noqa: E402


class Network(torch.nn.Module):
    """Embedding, residual FP8 blocks, norm; its output is the head's hidden state (BF16)."""

    def __init__(self, vocab, width, blocks):
        super().__init__()
        p = torch.nn.Parameter
        self.embed = p(torch.randn(vocab, width))
        self.up = torch.nn.ParameterList([p(torch.randn(2 * width, width) / width ** 0.5) for _ in range(blocks)])
        self.down = torch.nn.ParameterList([p(torch.randn(width, 2 * width) / (2 * width) ** 0.5)
                                            for _ in range(blocks)])
        self.head = p((torch.randn(vocab, width) * 0.02).to(torch.bfloat16))

    def forward(self, tokens):
        x = self.embed[tokens]
        for up, down in zip(self.up, self.down):
            h = fp8_linear(self.norm(x), up, activation="gelu")
            x = fp8_linear(h, down, residual=x, out_dtype=torch.float32)
        return self.norm(x)

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def train(steps=60, vocab=1000, width=192, blocks=2, tokens=600, seed=0, device="cuda"):
    """(network, losses, next token of each token) after ``steps`` of AdamW on random batches."""
    torch.manual_seed(seed)
    net = Network(vocab, width, blocks).to(device)
    after = torch.randperm(vocab, device=device)
    opt = torch.optim.AdamW(net.parameters(), lr=3e-3, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        x = torch.randint(0, vocab, (tokens,), device=device)
        mask = (torch.rand(tokens, device=device) < 0.9).to(torch.uint8)  # prompts and padding are not scored
        loss = linear_cross_entropy(net(x), net.head, after[x], mask, label_smoothing=0.05, z_loss=1e-4)
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return net, [float(v) for v in losses], after


@torch.no_grad()
def rollout_drift(net, after, count=8):
    """(logp of an 8-bit head, logp of the BF16 head, standard deviation of the logits) of ``count`` single tokens."""
    vocab, width = net.head.shape
    head_q, head_s = rlk.fp8_quantize(net.head, block_rows=128)  # once, as a server would keep it
    x = torch.arange(count, device=net.head.device)
    hidden, target = net(x), after[x]
    on = torch.ones(1, dtype=torch.uint8, device=hidden.device)
    rolled, spread = [], 0.0
    for i in range(count):  # one token at a time: the weight is read once a token
        logits = rlk.fp8_matmul(*rlk.fp8_quantize(hidden[i:i + 1]), head_q, head_s)
        c = rlk.Contract(T=1, V_real=vocab, V_padded=vocab, num_tiles=8)
        rolled.append(rlk.logp_fwd(c, logits, target[i:i + 1], on)[0])
        spread = max(spread, float(logits.float().std()))
    c = rlk.linear_ce_contract(hidden, net.head, on.expand(count).contiguous())
    nll, _ = rlk.linear_ce_fwd(c, hidden, net.head, target, on.expand(count).contiguous())
    return torch.cat(rolled), -nll, spread


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    net, losses, after = train(a.steps)
    for k in range(0, len(losses), max(1, len(losses) // 6)):
        print("step %4d  loss %.4f" % (k, losses[k]))
    print("last       loss %.4f" % losses[-1])
    rolled, trained, spread = rollout_drift(net, after)
    print("8-bit head against BF16 head: mean |logp difference| %.4f, largest %.4f (logits' deviation %.2f)" % (
        (rolled - trained).abs().mean(), (rolled - trained).abs().max(), spread))


if __name__ == "__main__":
    main()
