"""A learned-sparse-attention layer around the selection, run as it would be used.

Serving: the tokens of a prompt, then single tokens. Index keys and key / value rows
are rotated, quantised to e4m3 and written into their caches; each query selects its
exact top-k rows by the indexer scores and attends over those rows of the cache.

Training: the same selection on bf16 rows, the attention with its gradients, and the
gradients of rotated queries back through the rotation.

    python examples/sparse_attention.py [--context 65536] [--k 2048]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import exact_top_token_gb300 as hk  # noqa: E402


class Cache:
    """e4m3 rows with one fp32 scale per (row, head)."""

    def __init__(self, rows, heads, d, device):
        self.codes = torch.zeros(rows, heads, d, dtype=torch.uint8, device=device).view(
            torch.float8_e4m3fn)
        self.scale = torch.ones(rows, heads, device=device)

    def write(self, x, slots, positions=None, freq=None, mscale=1.0):
        hk.cache_write(x, self.codes, self.scale, slots=slots, positions=positions, inv_freq=freq,
                       mscale=mscale)


class Layer:
    """Random projections' outputs stand in for the projections of a model."""

    def __init__(self, context, k, heads=64, cache_heads=1, d=128, index_heads=64, seed=0,
                 device="cuda"):
        self.k, self.heads, self.index_heads, self.d = k, heads, index_heads, d
        self.gen = torch.Generator(device=device).manual_seed(seed)
        self.device = device
        # half of each row is rotated; frequencies scaled for a context past the original one.
        # The factor that goes with the table is on queries and keys, wherever they are rotated:
        # the rotated part of a score carries its square.
        self.freq, self.mscale = hk.rope_frequencies(d // 2, scaling="parts", factor=16.0,
                                                     original_context=4096, device=device)
        self.index_keys = Cache(context, 1, d, device)
        self.keys = Cache(context, cache_heads, d, device)
        self.values = Cache(context, cache_heads, d, device)
        self.cache_heads = cache_heads
        self.length = 0

    def _rows(self, n, heads):
        return torch.randn(n, heads, self.d, device=self.device, generator=self.gen).bfloat16()

    def append(self, n):
        """n new tokens into the caches; returns their positions."""
        slots = torch.arange(self.length, self.length + n, dtype=torch.int32, device=self.device)
        self.index_keys.write(self._rows(n, 1), slots, slots, self.freq, self.mscale)
        self.keys.write(self._rows(n, self.cache_heads), slots, slots, self.freq, self.mscale)
        self.values.write(self._rows(n, self.cache_heads), slots)
        self.length += n
        return slots

    def forward(self, positions):
        """Selects and attends for the queries at `positions`; returns (out, lse, idx)."""
        n = positions.numel()
        iq = torch.empty(n, self.index_heads, self.d, dtype=torch.uint8,
                         device=self.device).view(torch.float8_e4m3fn)
        iq_scale = torch.empty(n, self.index_heads, device=self.device)
        hk.cache_write(self._rows(n, self.index_heads), iq, iq_scale, positions=positions,
                       inv_freq=self.freq, mscale=self.mscale)
        w = torch.rand(n, self.index_heads, device=self.device, generator=self.gen)
        idx, _, _ = hk.select(iq, self.index_keys.codes[:self.length, 0], w, positions, self.k,
                              q_scale=iq_scale, k_scale=self.index_keys.scale[:self.length, 0])
        q = hk.rope(self._rows(n, self.heads), positions, self.freq, mscale=self.mscale)
        out, lse = hk.attend(q, self.keys.codes[:self.length], self.values.codes[:self.length], idx,
                             k_scale=self.keys.scale[:self.length],
                             v_scale=self.values.scale[:self.length])
        return out, lse, idx

    def train_step(self, positions, idx):
        """Attention over bf16 rows with gradients of the projections' outputs."""
        n = positions.numel()
        rows = torch.arange(self.length, dtype=torch.int32, device=self.device)
        x_q, x_k = self._rows(n, self.heads), self._rows(self.length, self.cache_heads)
        v = self._rows(self.length, self.cache_heads)
        q = hk.rope(x_q, positions, self.freq, mscale=self.mscale)
        k = hk.rope(x_k, rows, self.freq, mscale=self.mscale)
        out, lse = hk.attend(q, k, v, idx, out_dtype=torch.float32)
        grad = self._rows(n, self.heads)                       # of the loss with respect to out
        dq, dk, dv = hk.attend_backward(q, k, v, idx, out, lse, grad)
        # through the rotation
        dx_q = hk.rope(dq, positions, self.freq, mscale=self.mscale, inverse=True)
        dx_k = hk.rope(dk, rows, self.freq, mscale=self.mscale, inverse=True)
        return out, dx_q, dx_k, dv


def main(context=65536, k=2048, prompt=256, tokens=8):
    layer = Layer(context, k)
    layer.append(context - prompt - tokens)   # what the caches hold already
    positions = layer.append(prompt)
    out, lse, idx = layer.forward(positions)
    print(f"prompt: {prompt} queries over {layer.length} rows, out {tuple(out.shape)}, "
          f"mean lse {lse.mean().item():.3f}")
    for _ in range(tokens):
        out, lse, last = layer.forward(layer.append(1))
    print(f"decoded {tokens} tokens; the last one selected {int((last >= 0).sum())} rows")
    grads = layer.train_step(positions, idx)
    print("training step:", ", ".join(f"{g.float().norm().item():.4g}" for g in grads),
          "(norms of out, dq, dk, dv)")
    return out, grads


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--context", type=int, default=65536)
    ap.add_argument("--k", type=int, default=2048)
    ap.add_argument("--prompt", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args()
    main(a.context, a.k, a.prompt, a.tokens)
