"""A draft head on the library's operators: decoding with log probabilities,
greedy verification of the drafts, and a training step.

    python examples/draft_head.py [--rows 64] [--hidden 1024] [--vocab 50257] [--steps 20]

The head is  h = norm1(x);  b = h + silu(h W1^T + b1);  logits = norm2(b) Wv^T,
the logits' vocabulary cut into shards of whole columns.  Parameters and
activations are bf16 (or fp32); the norms' weights are fp32.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import vocab_argmax_amd as vpa


class DraftHead:
    def __init__(self, hidden, vocab, n_shards=2, dtype=torch.bfloat16, device="cuda:0", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.vocab, self.n_shards = vocab, n_shards
        self.shard_width = -(-vocab // n_shards)
        self.dtype, self.device = dtype, torch.device(device)

        def normal(*shape):
            return (torch.randn(shape, generator=g, device=device) * hidden ** -0.5).to(dtype)
        f32 = dict(dtype=torch.float32, device=device)
        self.params = {
            "norm1.weight": torch.ones(hidden, **f32), "norm1.bias": torch.zeros(hidden, **f32),
            "block.weight": normal(hidden, hidden), "block.bias": normal(hidden),
            "norm2.weight": torch.ones(hidden, **f32), "norm2.bias": torch.zeros(hidden, **f32),
            "vocab.weight": normal(vocab, hidden),
        }

    def forward(self, x, keep=False):
        """Logits [rows, vocab] of x's dtype; with keep, also what backward() takes."""
        p = self.params
        h, m1, r1 = vpa.layer_norm(x, p["norm1.weight"], p["norm1.bias"], with_stats=True)
        b = vpa.head_linear(h, p["block.weight"], p["block.bias"], "silu", residual=h,
                            with_pre=keep)
        b, pre = b if keep else (b, None)
        y, m2, r2 = vpa.layer_norm(b, p["norm2.weight"], p["norm2.bias"], with_stats=True)
        logits = vpa.head_linear(y, p["vocab.weight"])
        return (logits, (x, m1, r1, h, pre, b, m2, r2, y)) if keep else logits

    def decode(self, x, n_top=5):
        """Greedy tokens of each row, their log probabilities and the most
        likely alternatives -> (ids, TokenLogprobs)."""
        logits = self.forward(x)
        ids, _ = vpa.top_tokens(logits, self.vocab, self.shard_width, self.n_shards)
        return ids, vpa.token_logprobs(logits, self.vocab, self.shard_width, self.n_shards, ids,
                                       n_top)

    def verify(self, x, draft_ids):
        """Greedy verification of draft_ids [requests, K] for the rows x
        [requests * (K + 1), hidden] -> (out_tokens, num_sampled, num_rejected,
        target_ids, log probabilities of the target tokens)."""
        r, k = draft_ids.shape
        logits = self.forward(x)
        v, w, s = self.vocab, self.shard_width, self.n_shards
        out, sampled, rejected, targets = vpa.greedy_verify(
            *vpa.verify_stats(logits, v, w, s, r, k), draft_ids)
        lp = vpa.token_logprobs(logits, v, w, s, targets.view(-1)).logprobs.view(r, k + 1)
        return out, sampled, rejected, targets, lp

    def loss_and_grads(self, x, targets, entropy_weight=0.0):
        """Mean of -log p(target) - entropy_weight * entropy over the rows, its
        gradients by the parameters (of their dtypes) and by x.  Rows whose
        target is -1 count with their entropy only."""
        p = self.params
        v, w, s = self.vocab, self.shard_width, self.n_shards
        logits, (x, m1, r1, h, pre, b, m2, r2, y) = self.forward(x, keep=True)
        out = vpa.token_logprobs(logits, v, w, s, targets)
        n = x.shape[0]
        loss = -(out.logprobs.mean() + entropy_weight * out.entropy.mean())
        g_lp = torch.full((n,), -1.0 / n, device=self.device)
        g_ent = torch.full((n,), -entropy_weight / n, device=self.device) if entropy_weight else None
        # the logits are not needed after this: their gradient takes their place
        d = vpa.token_logprobs_backward(logits, v, w, s, targets, out.row_stats, g_lp, g_ent,
                                        out=logits)
        g = {}
        dy, g["vocab.weight"], _ = vpa.head_linear_backward(d, y, p["vocab.weight"],
                                                            need_bias=False)
        db, g["norm2.weight"], g["norm2.bias"] = vpa.layer_norm_backward(dy, b, m2, r2,
                                                                         p["norm2.weight"])
        dh, g["block.weight"], g["block.bias"] = vpa.head_linear_backward(
            db, h, p["block.weight"], pre, "silu")
        dh += db                                          # the block's residual
        dx, g["norm1.weight"], g["norm1.bias"] = vpa.layer_norm_backward(dh, x, m1, r1,
                                                                         p["norm1.weight"])
        return loss, g, dx

    def train_step(self, x, targets, lr, entropy_weight=0.0):
        loss, g, _ = self.loss_and_grads(x, targets, entropy_weight)
        for name, t in self.params.items():
            t.add_(g[name], alpha=-lr)
        return loss


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=50257)
    ap.add_argument("--shards", type=int, default=2)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.5)
    ap.add_argument("--fp32", action="store_true")
    args = ap.parse_args()
    dtype = torch.float32 if args.fp32 else torch.bfloat16
    head = DraftHead(args.hidden, args.vocab, args.shards, dtype)
    g = torch.Generator(device=head.device)
    g.manual_seed(1)
    x = torch.randn(args.rows, args.hidden, generator=g, device=head.device).to(dtype)
    targets = torch.randint(0, args.vocab, (args.rows,), generator=g, device=head.device,
                            dtype=torch.int32)
    for step in range(args.steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        loss = head.train_step(x, targets, args.lr).item()
        print(f"step {step:3d}  loss {loss:8.4f}  {1e3 * (time.perf_counter() - t0):7.2f} ms")
    ids, r = head.decode(x)
    print(f"decoded: {int((ids == targets).sum())} of {args.rows} rows give their target, "
          f"mean log probability {r.logprobs.mean().item():.4f}, "
          f"mean entropy {r.entropy.mean().item():.4f}")
    k = 3
    req = args.rows // (k + 1)
    if req:
        rows = x[:req * (k + 1)]
        drafts = targets[:req * (k + 1)].view(req, k + 1)[:, :k].contiguous()
        _, sampled, _, _, lp = head.verify(rows, drafts)
        print(f"verified: {sampled.float().mean().item():.2f} tokens a request of up to {k + 1}, "
              f"mean log probability of the targets {lp.mean().item():.4f}")


if __name__ == "__main__":
    main()
