"""Shared parts of the KV-cache tests: batches on the device with their
oracle, and the tolerances."""

from __future__ import annotations

import numpy as np
import torch

import weight_only_int4_gemv_b200 as awq
from oracle import kv_oracle as K

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def to64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def i32(values, device="cuda") -> torch.Tensor:
    return torch.tensor(values, dtype=torch.int32, device=device)


class Setup:
    """A cache of random pages handed out to sequences, on the device (cache)
    and in the oracle (ref)."""

    def __init__(self, max_lens, heads, dim, page, fmt, seed=0, spare=2, filled=True, layers=1):
        rng = np.random.default_rng(seed)
        self.rng, self.fmt, self.heads, self.dim, self.page = rng, fmt, heads, dim, page
        counts = [-(-m // page) for m in max_lens]
        n = sum(counts) + spare
        order = rng.permutation(n).astype(np.int32)
        self.table = np.zeros((len(max_lens), max(counts + [1])), np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.n_pages = n
        codes, scales = [], []
        for w in range(2):
            if filled:
                x = rng.standard_normal((n, heads, page // 16, 16, dim)) * (1.5 if w == 0 else 0.7)
                s = (np.abs(x).max((3, 4)) / K.TOP[fmt]).astype(np.float32)
                c = K.encode(x / s[..., None, None].astype(np.float64), fmt).reshape(n, heads, page, dim)
            else:        # whatever memory held before: any byte (NaN codes among e4m3's), any scale
                s = rng.choice(np.array([np.nan, np.inf, -1.0, 0.0, 1e30], np.float32), (n, heads, page // 16))
                c = rng.integers(0, 256, (n, heads, page, dim)).astype(np.uint8)
            codes.append(c)
            scales.append(s)
        self.ref = K.Cache(codes[0], codes[1], scales[0], scales[1], fmt)
        # the device pages: one layer's slice of an array that holds `layers` of them
        dev = []
        for a in codes + scales:
            t = torch.zeros((n, layers) + a.shape[1:], dtype=torch.uint8 if a.dtype == np.uint8 else torch.float32,
                            device="cuda")
            t[:, layers - 1] = torch.from_numpy(a).cuda()
            dev.append(t[:, layers - 1])
        self.cache = awq.KvCache(dev[0], dev[1], dev[2], dev[3], fmt)

    def batch(self, lens, new, max_q_len=None, table=None, wide=False):
        """wide: room for long sequences in the table (its unused entries name no page), which with more than 64 rows
        to a sequence and head makes the attention take its many-row kernel."""
        indptr = np.concatenate([[0], np.cumsum(new)])
        table = self.table if table is None else table
        if wide:
            table = np.concatenate([table, np.full((len(table), 40000 // self.page), -1, np.int32)], 1)
        return awq.KvBatch(torch.from_numpy(table).cuda(), i32(lens), i32(indptr), max_q_len)

    def poison(self, lens):
        """Blocks behind each sequence's last one get NaN scales and bytes; so do the bytes behind its end."""
        for b, n in enumerate(lens):
            for pos in range(n, self.table.shape[1] * self.page):
                if pos // self.page >= -(-max(n, 1) // self.page):
                    break
                pg, off = int(self.table[b, pos // self.page]), pos % self.page
                for pages, scales in ((self.cache.k_pages, self.cache.k_scales),
                                      (self.cache.v_pages, self.cache.v_scales)):
                    pages[pg, :, off] = 0xFF
                    if off // 16 * 16 >= n - pos + off:
                        scales[pg, :, off // 16] = float("nan")

    def expect(self, q, lens, new, scale=None, window=0, sinks=0, keep=None):
        """Oracle outputs and the elementwise tolerance for q [tokens, heads, dim] (float64). keep: for each sequence
        which of its keys are there (None: all)."""
        scale = self.dim ** -0.5 if scale is None else scale
        out, tol, at = np.zeros_like(q), np.zeros_like(q), 0
        for b, (n, a) in enumerate(zip(lens, new)):
            k = self.ref.values(0, self.table[b], 0, n)
            v = self.ref.values(1, self.table[b], 0, n)
            top = self.ref.tops(1, self.table[b], 0, n)
            y, mass, big, small = K.attention(q[at:at + a], k, v, n - a, scale, window, sinks, top,
                                              None if keep is None else keep[b])
            out[at:at + a] = y
            # Weights rounded to fp16 (half a step: 2^-11) move y by 2^-11 sum w |v|. Below fp16's normal range the
            # error is 2^-25 against a largest weight of at least 1, weights there being w times the value scale:
            # 2^-25 n max(w top). A logit off by d moves each weight by a factor 1 +- d, so y by 2 d sum w |v|:
            # 8 steps of 17 additions in fp32 that may truncate, 136 * 2^-24 < 2^-16 of sum |q| |k|, and the scale,
            # log2 and exp2 in fp32 of logits below 100 in log2 units: 2^-17.
            d = 2.0 ** -16 * big + 2.0 ** -17
            tol[at:at + a] = (2.0 ** -11 + 2 * d[..., None]) * mass + 2.0 ** -25 * small[..., None]
            at += a
        return out, tol


def check(got: torch.Tensor, want: np.ndarray, tol: np.ndarray, tag=""):
    """|got - want| within tol plus half a step of got's type."""
    half = torch.finfo(got.dtype).eps / 2
    y = to64(got)
    assert np.isfinite(y).all(), f"{tag}: non-finite output"
    over = np.abs(y - want) - (tol + half * (np.abs(want) + tol) + 2.0 ** -25)
    assert over.max(initial=-1.0) <= 0, f"{tag}: {over.max():.3e} over the tolerance, at {np.argwhere(over > 0)[:4].tolist()}"
