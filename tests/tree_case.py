"""Seeded drafted-token batches over a paged cache, on the host and on the device, for the tree tests."""
from __future__ import annotations

import random
from typing import List, Optional, Sequence

import numpy as np
import torch

import paged_kv_cache_385_b200 as pa
from oracle import tree

KV = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
QD = {"f16": torch.float16, "bf16": torch.bfloat16}


def random_masks(counts: Sequence[int], seed: int) -> List[int]:
    """A random tree per sequence, node 0 its root: each node's ancestors and itself, as bits."""
    r = random.Random(seed)
    rows = []
    for n in counts:
        seen = []
        for i in range(n):
            seen.append((seen[r.randrange(max(0, i - 9), i)] if i else 0) | 1 << i)
        rows += seen
    return rows


def mask_words(masks: Sequence[int], words: int) -> torch.Tensor:
    full = (1 << 64) - 1
    rows = [[m >> 64 * w & full for w in range(words)] for m in masks]
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in rows], dtype=torch.int64).reshape(-1, words)


class TreeCase:
    """A batch whose pools hold seeded values; pages in a seeded order, unused ones and rows NaN or random bits."""

    def __init__(self, kv: str, d: int, hkv: int, group: int, counts: Sequence[int], lens: Sequence[int], *, q: str = "",
                 masks="tree", softcap: float = 0.0, seed: int = 1, extra_rows: int = 0, order: Optional[int] = None,
                 scale: Optional[float] = None):
        self.kv, self.d, self.hkv, self.hq = kv, d, hkv, hkv * group
        self.counts, self.lens_host, self.softcap = list(counts), list(lens), softcap
        self.scale = d ** -0.5 if scale is None else scale
        self.k_scale, self.v_scale = (0.02, 0.03) if kv == "e4m3" else (1.0, 1.0)
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // 16) for n in lens]
        self.num_blocks = sum(need) + 3
        ids = torch.randperm(self.num_blocks, generator=torch.Generator().manual_seed(seed if order is None else order))
        self.bt_host = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for s, k in enumerate(need):
            self.bt_host[s, :k] = ids[at:at + k].to(torch.int32)
            at += k
        self.pools = []
        for scale_ in (self.k_scale, self.v_scale):
            # Every row a NaN first: rows behind a context, and pages of nobody, may hold anything.
            pool = torch.full((self.num_blocks, hkv, 16, d), float("nan")).to(KV[kv])
            for s, n in enumerate(lens):
                rows = (torch.randn(n, hkv, d, generator=g) / scale_).clamp(-448, 448).to(KV[kv])
                t = torch.arange(n)
                pool.view(torch.uint8 if kv == "e4m3" else torch.int16)[self.bt_host[s, t // 16].long(), :, t % 16] = \
                    rows.view(torch.uint8 if kv == "e4m3" else torch.int16)
            self.pools.append(pool)
        self.start_host = [0]
        for n in counts:
            self.start_host.append(self.start_host[-1] + n)
        T = self.start_host[-1] + extra_rows
        self.qt = QD[q or (kv if kv != "e4m3" else "bf16")]
        self.q_host = torch.randn(T, self.hq, d, generator=g).to(self.qt)
        self.masks = random_masks(counts, seed) if masks == "tree" else masks
        self.words = max(1, -(-max(list(counts) + [1]) // 64))

    def host_pool(self, which: int) -> np.ndarray:
        p = self.pools[which]
        return p.view(torch.uint8).reshape(*p.shape[:3], -1).numpy()

    def oracle(self):
        return tree.attend_paged(self.q_host.double().numpy(), self.host_pool(0), self.host_pool(1),
                                 self.bt_host.numpy(), self.start_host, self.lens_host, self.masks, self.scale,
                                 self.hkv, self.kv, self.softcap, self.k_scale, self.v_scale)

    def to_device(self):
        self.k_cache, self.v_cache = (p.cuda() for p in self.pools)
        self.bt = self.bt_host.cuda()
        self.start = torch.tensor(self.start_host, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(self.lens_host, dtype=torch.int32, device="cuda")
        self.q = self.q_host.cuda()
        extra = self.q_host.shape[0] - self.start_host[-1]
        self.mask = None if self.masks is None else mask_words(list(self.masks) + [0] * extra, self.words).cuda()
        self.out = torch.full_like(self.q, 77.0)
        return self

    def workspace(self, fill: int = 0xff):
        n = pa.pa_decode_tree_workspace_bytes(len(self.lens_host), self.hq, self.hkv, self.d, max(self.counts),
                                              max(self.lens_host))
        return torch.full((n,), fill, dtype=torch.uint8, device="cuda") if n else None

    def run(self, out: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None, **kw) -> torch.Tensor:
        out = self.out if out is None else out
        kw = {"max_context_len": max(self.lens_host), "workspace": self.workspace(), **kw}
        pa.pa_decode_tree(out, self.q if q is None else q, self.k_cache, self.v_cache, self.bt, self.start, self.lens,
                          self.mask, max(self.counts), self.scale, self.hkv, softcap=self.softcap,
                          k_scale=self.k_scale, v_scale=self.v_scale, **kw)
        return out

    def bound(self, out: np.ndarray, weight: np.ndarray) -> np.ndarray:
        """How far a right kernel may be from the exact row, by its roundings (u half a step, relative).

        A softmax weight is rounded to the products' 16-bit type: u_p of it, so u_p * sum w |V|; the row's
        result to q's type: u_o |out|. A score in float32 is off by at most (D + 2) 2^-24 sum |q k| scale;
        with |q|, |k| ~ N(0, 1) and scale 1/sqrt(D) that is below 2^-15 for D <= 128 (sum |q k| <= 2 D, and
        the capped form adds a few 2^-22 of the cap), which moves a weight by that much, relative; so do the
        float32 sums over the keys (2^-24 each, random in sign) and the 2^-22 of the base-2 exponential:
        2^-13 of sum w |V| covers the four."""
        u_p = 2.0 ** -8 if self.kv == "bf16" else 2.0 ** -11
        u_o = 2.0 ** -8 if self.qt == torch.bfloat16 else 2.0 ** -11
        return (u_p + 2.0 ** -13) * weight + u_o * np.abs(out) * (1 + 2.0 ** -7) + 2.0 ** -24
