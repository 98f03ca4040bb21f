"""Plain fp64 numpy form of the 8-bit page format (include/gdn_attn.h), written from its definition
alone, and the caches that its tests share.  What a row sees and attention itself are
attention_ref's."""
from __future__ import annotations

import numpy as np
import torch

from tests import attention_ref as R

GRID = R.e4m3(np.arange(127))                 # ascending, of even index where the code is even
MOST_E = 22


def exponent_at(page_size, d, which, row):
    """Byte of a block with the exponent of a row's keys (0) or values (1)."""
    return 2 * page_size * d + 16 * (row // 128) + 8 * which + row % 128 // 16


def page_bytes(page_size, d):
    return 2 * page_size * d + 16 * max(1, page_size // 128)


def least_exponent(m):
    """The least exponent under which magnitude m is at most 448."""
    return np.minimum(np.searchsorted(448.0 * 2.0 ** np.arange(-15.0, 8.0), m), MOST_E)


def nearest(x):
    """The nearest e4m3 number, at most 448, ties to the even code: its magnitude's code."""
    a = np.minimum(np.abs(x), 448.0)
    i = np.clip(np.searchsorted(GRID, a), 1, 126)
    low, high = a - GRID[i - 1], GRID[i] - a
    return np.where((high < low) | ((high == low) & (i % 2 == 0)), i, i - 1)


def block(pages, page, h, page_size, d):
    """Keys and values [page_size, d] of one (page, head), without the head's scales."""
    raw = pages[page, h]
    out = []
    for i in (0, 1):
        v = R.e4m3(raw[i * page_size * d:(i + 1) * page_size * d].reshape(page_size, d))
        e = np.array([raw[exponent_at(page_size, d, i, r)] for r in range(page_size)], dtype=np.float64)
        with np.errstate(over="ignore", invalid="ignore"):
            out.append(v * 2.0 ** (e - 15)[:, None])
    return out


def cached(pages, table, length, H, page_size, d, head_scale=None):
    """Keys and values [H, length, d] of one sequence."""
    k, v = np.zeros((2, H, length, d))
    for p in range(-(-length // page_size)):
        n = min(page_size, length - p * page_size)
        for h in range(H):
            a, b = block(pages, table[p], h, page_size, d)
            k[h, p * page_size:p * page_size + n] = a[:n]
            v[h, p * page_size:p * page_size + n] = b[:n]
    if head_scale is not None:
        k *= head_scale[0][:, None, None]
        v *= head_scale[1][:, None, None]
    return k, v


class Cache8:
    """A cache of random codes and exponents, as a kernel and as numpy see it: `lens` tokens in
    each sequence, pages in random order, everything outside the sequences 0xFF (NaN codes, and
    exponents that no block has)."""

    def __init__(self, lens, H, page_size, d, *, new=None, head_scale=False, seed=0, spare=2,
                 exponents=(3, 9)):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.page_size, self.d = list(lens), H, page_size, d
        self.new = list(new) if new is not None else [1] * len(lens)
        counts = [-(-n // page_size) for n in lens]
        total = sum(counts) + spare
        order = rng.permutation(total)
        pages = np.full((total, H, page_bytes(page_size, d)), 255, dtype=np.uint8)
        self.table = np.full((len(lens), max(1, max(counts, default=1))), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(lens):
            for p in range(counts[b]):
                page = order[at]
                at += 1
                self.table[b, p] = page
                m = min(page_size, n - p * page_size)
                for i in (0, 1):
                    x = rng.integers(0, 127, (H, m * d)) + 128 * rng.integers(0, 2, (H, m * d))
                    pages[page, :, i * page_size * d:i * page_size * d + m * d] = x
                    for r in range(0, m, 16):
                        pages[page, :, exponent_at(page_size, d, i, r)] = rng.integers(
                            exponents[0], exponents[1] + 1, H)
        self.np_pages = pages
        self.scale = (0.25 + rng.random((2, H))).astype(np.float32) if head_scale else None
        self.table_t = torch.from_numpy(self.table).cuda()
        self.len_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.at = np.concatenate([[0], np.cumsum(self.new)])
        self.cu = torch.tensor(self.at, dtype=torch.int32, device="cuda")
        self.scale_t = None if self.scale is None else torch.from_numpy(self.scale).cuda()
        self.upload()

    def upload(self):
        self.pages = torch.from_numpy(self.np_pages).cuda()

    @property
    def tokens(self):
        return int(self.at[-1])

    def reference(self, q, scale, causal, window):
        """attention() of every sequence, the rows packed again."""
        out = [np.zeros(q.shape), np.full(q.shape[:2], -np.inf), np.zeros(q.shape),
               np.zeros(q.shape[:2])]
        for b, n in enumerate(self.lens):
            k, v = cached(self.np_pages, self.table[b], n, self.H, self.page_size, self.d,
                          None if self.scale is None else self.scale.astype(np.float64))
            sl = slice(self.at[b], self.at[b + 1])
            for whole, part in zip(out, R.attention(q[sl], k, v, n, scale, causal, window)):
                whole[sl] = part
        return out
