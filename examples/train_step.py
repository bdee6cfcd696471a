"""A small decoder trained reproducibly: embedding lookup, layer norm, attention over packed documents with capped scores and
shared key heads, the exact cross-entropy, and AdamW with 8-bit states, as one training program.

    python examples/train_step.py [--steps 20] [--state-bits 8]

Trains twice from the same seed and checks that every parameter, optimizer state and loss is equal byte for
byte.  Products with weight matrices are torch.matmul (cuBLAS, with its reproducible workspace setting).
"""
import argparse
import math
import os
import sys

os.environ.setdefault("CUBLAS_WORKSPACE_CONFIG", ":4096:8")

import torch  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bitwise_deterministic_shard_gb300 as da  # noqa: E402


class Decoder:
    """Pre-norm decoder in bf16 with f32 norm weights; the output projection is the embedding."""

    def __init__(self, vocab=512, width=256, heads=8, kv_heads=2, layers=2, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.width, self.heads, self.kv_heads, self.head = width, heads, kv_heads, width // heads

        def matrix(n, m, scale):
            return (torch.randn(n, m, generator=g) * scale).to(device, torch.bfloat16).requires_grad_(True)

        def norm():
            return [torch.ones(width, device=device, requires_grad=True), torch.zeros(width, device=device, requires_grad=True)]
        s = 1 / math.sqrt(width)
        self.embedding = matrix(vocab, width, 0.02)
        self.layers = [{"norm1": norm(), "qkv": matrix((heads + 2 * kv_heads) * self.head, width, s),
                        "out": matrix(width, width, s / math.sqrt(2 * layers)), "norm2": norm(),
                        "up": matrix(4 * width, width, s), "down": matrix(width, 4 * width, 0.5 * s / math.sqrt(2 * layers))}
                       for _ in range(layers)]
        self.norm = norm()

    def parameters(self):
        ps = [self.embedding, *self.norm]
        for layer in self.layers:
            for v in layer.values():
                ps += v if isinstance(v, list) else [v]
        return ps

    def loss(self, tokens, targets, docs):
        """Mean loss of [B, S] targets; docs: document of each token (attention stays within one)."""
        B, S = tokens.shape
        x = da.embedding(tokens, self.embedding)
        for p in self.layers:
            q, k, v = (da.layer_norm(x, *p["norm1"]) @ p["qkv"].mT).split(
                [self.heads * self.head, self.kv_heads * self.head, self.kv_heads * self.head], -1)
            q, k, v = (t.view(B, S, -1, self.head).transpose(1, 2) for t in (q, k, v))    # views: nothing is copied
            a = da.attention(q, k, v, causal=True, softcap=30.0, docs=docs)
            x = x + a.transpose(1, 2).reshape(B, S, -1) @ p["out"].mT
            x = x + torch.nn.functional.gelu(da.layer_norm(x, *p["norm2"]) @ p["up"].mT) @ p["down"].mT
        logits = (da.layer_norm(x, *self.norm) @ self.embedding.mT).view(B * S, -1)
        return da.cross_entropy(logits, targets.reshape(-1))


def batch(step, B=4, S=384, vocab=512, device="cuda"):
    """Packed documents of a synthetic language (each token follows from the one before), padded at the end."""
    g = torch.Generator().manual_seed(1000 + step)
    x = torch.randint(0, vocab, (B, S + 1), generator=g)
    for t in range(1, S + 1):
        keep = torch.rand(B, generator=g) < 0.9
        x[:, t] = torch.where(keep, (x[:, t - 1] * 7 + 3) % vocab, x[:, t])
    docs = (torch.arange(S) * 3 // S).repeat(B, 1).int()
    docs[:, -5:] = -1
    return x[:, :-1].to(device), x[:, 1:].to(device), docs.to(device)


def train(steps=20, state_bits=8, seed=0):
    """(losses, parameters, optimizer states) of a training run."""
    model = Decoder(seed=seed)
    opt = da.AdamW(model.parameters(), lr=3e-3, betas=(0.9, 0.95), weight_decay=0.1, state_bits=state_bits)
    losses = []
    for i in range(steps):
        loss = model.loss(*batch(i))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    states = [t for g in opt.groups for k, t in g.items() if k != "params"]
    return torch.stack(losses), [p.detach() for p in model.parameters()], states


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    args = ap.parse_args()
    first, again = (train(args.steps, args.state_bits) for _ in range(2))
    for i, l in enumerate(first[0].tolist()):
        print(f"step {i:3d}  loss {l:.6f}")
    same = all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
               for a, b in zip(first, again) for x, y in zip(a if isinstance(a, list) else [a], b if isinstance(b, list) else [b]))
    print("two runs are equal byte for byte" if same else "two runs DIFFER")
    return 0 if same else 1


if __name__ == "__main__":
    raise SystemExit(main())
