"""Plain fp64 numpy forms of the attention layer (include/gdn_attn.h), written
from its definitions alone: rotary positions, the 4-bit page format, attention
over places that a row sees.  Also the inputs that its tests share."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def e4m3(byte):
    b = np.asarray(byte, dtype=np.int64)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e == 0, m / 512.0, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def rotate(x, cos, sin, pos, axes, adjacent, back=False):
    """x [..., tokens, d]; pos [n_axes, tokens]; cos, sin [positions, d_rot / 2]."""
    y = np.array(x, dtype=np.float64)
    half = cos.shape[1]
    for i in range(half):
        p = pos[axes[i]]
        c, s = cos[p, i], sin[p, i]
        if back:
            s = -s
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def block(pages, page, h, page_size, d):
    """Keys and values [page_size, d] of one (page, head), without the head's scales."""
    raw = pages[page, h].astype(np.int64)
    out = []
    for i in (0, 1):
        codes = raw[i * page_size * d // 2:(i + 1) * page_size * d // 2].reshape(page_size, d // 2)
        at = page_size * d + i * page_size * d // 16
        scale = e4m3(raw[at:at + page_size * d // 16].reshape(page_size, d // 16))
        v = np.empty((page_size, d))
        v[:, 0::2] = E2M1[codes & 15]
        v[:, 1::2] = E2M1[codes >> 4]
        out.append(v * np.repeat(scale, 16, axis=1))
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


def attention(q, k, v, length, scale, causal, window):
    """q [n, Hq, d] of one sequence, k, v [H, length, d]: (o, lse, weight of |v|, largest sum of
    |q_i k_i| scale), the last two for bounds on rounding."""
    n, Hq, d = q.shape
    G = Hq // k.shape[0] if k.shape[0] else 1
    o, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    mass, size = np.zeros((n, Hq, d)), np.zeros((n, Hq))
    for j in range(n):
        p = length - n + j
        hi = 0 if p < 0 else p + 1 if causal else length
        lo = max(0, p + 1 - window) if window else 0
        if hi <= lo:
            continue
        for i in range(Hq):
            kk, vv = k[i // G, lo:hi], v[i // G, lo:hi]
            s = kk @ q[j, i] * scale
            w = np.exp(s - np.max(s))
            lse[j, i] = np.max(s) + np.log(np.sum(w))
            w = w / np.sum(w)
            o[j, i] = w @ vv
            mass[j, i] = w @ np.abs(vv)
            size[j, i] = np.max(np.abs(kk) @ np.abs(q[j, i])) * abs(scale)
    return o, lse, mass, size


class Cache:
    """A cache of random codes and scales, as a kernel and as numpy see it: `lens` tokens in each
    sequence, pages in random order, everything outside the sequences 0xFF (NaN scales)."""

    def __init__(self, lens, H, page_size, d, *, new=None, head_scale=False, seed=0, spare=2):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.page_size, self.d = list(lens), H, page_size, d
        self.new = list(new) if new is not None else [1] * len(lens)
        counts = [-(-n // page_size) for n in lens]
        total = sum(counts) + spare
        order = rng.permutation(total)
        size = page_size * d * 9 // 8
        pages = np.full((total, H, size), 255, dtype=np.uint8)
        self.table = np.full((len(lens), max(1, max(counts, default=1))), -1, dtype=np.int32)
        at = 0
        code, scale = page_size * d // 2, page_size * d // 16
        for b, n in enumerate(lens):
            for p in range(counts[b]):
                page = order[at]
                at += 1
                self.table[b, p] = page
                m = min(page_size, n - p * page_size)
                for part, w in ((0, d // 2), (code, d // 2), (2 * code, d // 16),
                                (2 * code + scale, d // 16)):
                    x = rng.integers(0, 256, (H, m * w), dtype=np.uint8) if w == d // 2 else \
                        rng.integers(0x20, 0x40, (H, m * w), dtype=np.uint8)
                    pages[page, :, part:part + m * w] = x
        self.np_pages = pages
        self.scale = None
        if head_scale:
            self.scale = (0.25 + rng.random((2, H))).astype(np.float32)
        self.pages = torch.from_numpy(pages).cuda()
        self.table_t = torch.from_numpy(self.table).cuda()
        self.len_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        cu = np.concatenate([[0], np.cumsum(self.new)])
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.at = cu
        self.scale_t = None if self.scale is None else torch.from_numpy(self.scale).cuda()

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
            for whole, part in zip(out, attention(q[sl], k, v, n, scale, causal, window)):
                whole[sl] = part
        return out


def tolerance(ref, dtype):
    """Bounds on |o - o64|, from the roundings alone.

    bf16 rows: a probability is rounded to fp16 (2^-11 of itself; the sum that divides uses the
    unrounded ones) and o to bf16 (2^-9 of itself).  fp32 rows: both fp16 parts of q and of p
    leave 2^-22 of them.  Either way the score's fp32 sum over d products is off by at most some
    2^-22 of the sum of their magnitudes (and by the exponential's 2^-22), which moves
    every weight by that much.  Twice the sum of these, and 2^-126 for what underflows."""
    o, _, mass, size = ref
    weights = 2.0 ** -20 * (2 + size[..., None])
    if dtype == torch.bfloat16:
        return 2 * (mass * (2.0 ** -11 + weights) + np.abs(o) * 2.0 ** -9) + 2.0 ** -126
    return 2 * (mass * (2.0 ** -21 + weights) + np.abs(o) * 2.0 ** -24) + 2.0 ** -126
