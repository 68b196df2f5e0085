"""A small click model on the library: looked-up rows through one gated block per feature table.

Each sample has one ID for each of ``tables`` features.  A step

1. looks the IDs up in a merged table (absent ones are inserted);
2. groups the rows by feature table;
3. norms them with their table's parameters, keeping the input in 8 bits;
4. projects them twice with their table's matrices;
5. norms the first projection, gates it with the second, adds it to the rows
   (a residual block, its inputs kept in 8 bits);
6. scores a sample by the mean of its rows, and runs all of it backwards: the
   table's rows by Adam, the blocks' parameters by plain gradient descent.

    python examples/feature_blocks.py --samples 65536 --steps 20
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import hash_table_lookup_amd as htl  # noqa: E402


class FeatureBlocks:
    """One gated block per feature table over a merged embedding table (fp32 rows, bf16 products)."""

    def __init__(self, tables: int, dim: int, capacity_log2: int = 20, seed: int = 0, lr: float = 0.05):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.tables, self.dim, self.lr = tables, dim, lr
        self.table = htl.Table(capacity_log2, dim, "f32", init_seed=seed, adam=True)
        ones = torch.ones(tables, dim, device="cuda")
        self.before = [ones.clone(), torch.zeros_like(ones)]          # weight and bias of the norms
        self.after = [ones.clone(), torch.zeros_like(ones)]
        self.wz, self.wu = (torch.randn(tables, dim, dim, device="cuda", generator=gen) / dim ** 0.5 for _ in range(2))
        self.head = torch.randn(dim, device="cuda", generator=gen)
        self.kw = dict(kind="layer", eps=1e-6)
        self.steps = 0

    def _groups(self, samples: int) -> htl.RowGroups:
        """The plan for sample-major rows; a program with one batch size makes it once."""
        ids = (torch.arange(samples * self.tables, device="cuda") % self.tables).to(torch.int32)
        return htl.group_rows(ids, self.tables)

    def _blocks(self, x, groups, save: bool):
        h, kept = htl.norm_rows(x, *self.before, groups=groups, out_dtype="bf16", save="i8" if save else None, **self.kw)
        z = htl.grouped_mm(h, self.wz.bfloat16(), groups)
        u = htl.grouped_mm(h, self.wu.bfloat16(), groups)
        out, kept_z, kept_u = htl.norm_gate(x, z, u, *self.after, groups=groups, act="silu",
                                            save="e4m3" if save else None, **self.kw)
        return out, (h, kept, kept_z, kept_u)

    def _logits(self, out, samples: int):
        return out.view(samples, self.tables, self.dim).mean(1) @ self.head

    def score(self, keys: torch.Tensor) -> torch.Tensor:
        """Logits of samples; keys int64 [samples, tables]."""
        x = htl.lookup(self.table, keys.reshape(-1), step=self.steps)[0]
        return self._logits(self._blocks(x, self._groups(keys.shape[0]), False)[0], keys.shape[0])

    def step(self, keys: torch.Tensor, labels: torch.Tensor):
        """One training step; returns (the loss, the logits before it)."""
        samples = keys.shape[0]
        self.steps += 1
        x, unique, inverse, n_unique, slots, _ = htl.lookup(self.table, keys.reshape(-1), step=self.steps)
        groups = self._groups(samples)
        out, (h, kept, kept_z, kept_u) = self._blocks(x, groups, True)
        logits = self._logits(out, samples)
        loss = torch.nn.functional.binary_cross_entropy_with_logits(logits, labels)

        dlogits = (torch.sigmoid(logits) - labels) / samples
        pooled = out.view(samples, self.tables, self.dim).mean(1)
        dout = (dlogits[:, None] * self.head / self.tables).repeat_interleave(self.tables, 0)
        dz, du, *dafter = htl.norm_gate_backward(dout, kept_z, kept_u, *self.after, groups=groups, act="silu", **self.kw)
        dh, dwz = htl.grouped_mm_backward(dz, h, self.wz.bfloat16(), groups, dx_dtype="f32")
        dh_u, dwu = htl.grouped_mm_backward(du, h, self.wu.bfloat16(), groups, dx_dtype="f32")
        dx, *dbefore = htl.norm_rows_backward(dh.add_(dh_u), kept, self.before[0], groups=groups, bias=True,
                                              dresidual=dout, **self.kw)
        htl.segment_sum_adam(self.table, slots, dx, inverse, n_unique, unique.numel(), lr=self.lr, step=self.steps)
        for p, g in zip(self.before + self.after + [self.wz, self.wu, self.head],
                        dbefore + dafter + [dwz, dwu, pooled.t() @ dlogits]):
            p.sub_(g, alpha=self.lr)
        return loss, logits


def main():
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--samples", type=int, default=65536)
    a.add_argument("--tables", type=int, default=26)
    a.add_argument("--dim", type=int, default=128)
    a.add_argument("--steps", type=int, default=20)
    a.add_argument("--lr", type=float, default=0.01)
    a = a.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = torch.arange(a.tables, device="cuda") << 48
    keys = torch.randint(0, 10000, (a.samples, a.tables), device="cuda", generator=gen) | table
    labels = (keys[:, 0] % 3 == 0).float()
    model = FeatureBlocks(a.tables, a.dim, lr=a.lr)
    for i in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        loss, _ = model.step(keys, labels)
        torch.cuda.synchronize()
        print(f"step {i}: loss {loss.item():.4f}, {(time.perf_counter() - t) * 1e3:.2f} ms", flush=True)


if __name__ == "__main__":
    main()
