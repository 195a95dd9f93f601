"""Plain CPU reference of the resident 8-bit cache, for its tests: the write
rules in the binary32 roundings that define them (numpy), reads and attention
in 64 bits.  It shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

F32 = np.float32
TOP = {"FP8_DYNAMIC": 448.0, "INT8": 127.0}
TORCH_CODE = {"FP8_DYNAMIC": torch.float8_e4m3fn, "INT8": torch.int8}


def rule(amax, codec):
    a = np.maximum(np.asarray(amax, F32), F32(1e-12))
    return a * (F32(1) / F32(448)) if codec == "FP8_DYNAMIC" else a / F32(127)


def quantise(x, scale, codec):
    """uint8 codes of float32 x; NaN -> 0, infinities -> the largest code."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        t = np.asarray(x, F32) / F32(scale)
    t = np.where(np.isnan(t), F32(0), t)
    if codec == "INT8":
        return np.clip(np.rint(t), -127, 127).astype(np.int8).view(np.uint8)
    t = np.clip(t, F32(-448), F32(448)).astype(F32)
    return torch.from_numpy(np.ascontiguousarray(t)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def values(codes, codec):
    """float32 values of uint8 codes."""
    t = torch.from_numpy(np.ascontiguousarray(codes))
    return t.view(TORCH_CODE[codec]).float().numpy()


class Pool:
    """The cache on the host: codes as uint8, K and V both [P, H, T, D]."""

    def __init__(self, pages, heads, tokens, dim, codec, seed=0):
        r = np.random.default_rng(seed)
        self.codec, self.T = codec, tokens
        # whatever lay in the memory before: every byte value, scales of all kinds
        self.k, self.v = (r.integers(0, 256, (pages, heads, tokens, dim), dtype=np.uint8) for _ in range(2))
        self.ks, self.vs = (r.choice(np.array([0, 1, -3, np.nan, np.inf, 1e-3], F32), (pages, heads)) for _ in range(2))

    def tensors(self, device):
        dt = TORCH_CODE[self.codec]
        k = torch.from_numpy(self.k.copy()).to(device).view(dt)
        v = torch.from_numpy(np.ascontiguousarray(self.v.transpose(0, 1, 3, 2))).to(device).view(dt)
        return k, v, torch.from_numpy(self.ks.copy()).to(device), torch.from_numpy(self.vs.copy()).to(device)

    def write(self, table, cu, lengths, k, v):
        """k, v: float32 [rows, H, D].  Returns the sequences that held a value that is not finite."""
        odd = set()
        for b in range(len(lengths)):
            n, length = cu[b + 1] - cu[b], lengths[b]
            start = length - n
            first = max(start, 0)
            if n == 0:
                continue
            for i in range(first // self.T, -(-length // self.T)):
                s0, s1 = max(first, i * self.T), min(length, (i + 1) * self.T)
                page, q0, q1 = table[b][i], s0 - i * self.T, s1 - i * self.T
                for codes, scales, x in ((self.k, self.ks, k), (self.v, self.vs, v)):
                    new = x[cu[b] + s0 - start:cu[b] + s1 - start]                  # [n, H, D]
                    for h in range(codes.shape[1]):
                        y = new[:, h]
                        fin = np.isfinite(y)
                        if not fin.all():
                            odd.add(b)
                        need = rule(np.abs(np.where(fin, y, F32(0))).max(), self.codec)
                        old = scales[page, h]
                        if q0 == 0:
                            s = need
                        else:
                            usable = 0 < old < np.inf
                            s = max(old, need) if usable else need
                            if s != old:
                                was = values(codes[page, h, :q0], self.codec)
                                with np.errstate(invalid="ignore"):
                                    was = was * (old if usable else F32(0))
                                codes[page, h, :q0] = quantise(was, s, self.codec)
                        scales[page, h] = s
                        codes[page, h, q0:q1] = quantise(y, s, self.codec)
        return odd

    def rows64(self, table_row, length):
        """K and V values of positions [0, length), float64 [length, H, D]."""
        pos = np.arange(length)
        page, at = np.asarray(table_row)[pos // self.T], pos % self.T
        out = []
        for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
            out.append(values(codes[page, :, at], self.codec).astype(np.float64) * scales[page].astype(np.float64)[..., None])
        return out

    def v_scales64(self, table_row, length):
        """[length, H]: the V scale of each position's page."""
        return self.vs[np.asarray(table_row)[np.arange(length) // self.T]].astype(np.float64)

    def read(self, table, cu, lengths, n_rows, dtype):
        """Rows as the library rounds them: binary32 product, then the type."""
        H, D = self.k.shape[1], self.k.shape[3]
        out = [np.zeros((n_rows, H, D), F32) for _ in range(2)]
        for b in range(len(lengths)):
            n, length = cu[b + 1] - cu[b], lengths[b]
            pos = np.arange(max(length - n, 0), length)
            if not len(pos):
                continue
            page, at = np.asarray(table[b])[pos // self.T], pos % self.T
            for o, codes, scales in ((out[0], self.k, self.ks), (out[1], self.v, self.vs)):
                o[cu[b] + pos - (length - n)] = values(codes[page, :, at], self.codec) * scales[page][..., None]
        return [torch.from_numpy(o).to(dtype) for o in out]


def attend(pool, table, cu, lengths, q, scale, causal, window, hidden_pages=()):
    """float64 [rows, Hq, D] outputs, lse, and per element how far a result may
    be off before its own last rounding (see tolerance)."""
    n_rows, Hq, D = q.shape
    H = pool.k.shape[1]
    G = Hq // H
    out, lse, off = np.zeros((n_rows, Hq, D)), np.full((n_rows, Hq), -np.inf), np.zeros((n_rows, Hq, D))
    lse_off = np.zeros((n_rows, Hq))
    for b in range(len(lengths)):
        n, length = cu[b + 1] - cu[b], lengths[b]
        if n == 0 or length == 0:
            continue
        pages = np.where(np.isin(np.arange(len(table[b])), hidden_pages), 0, table[b])
        K, V = pool.rows64(pages, length)
        S = pool.v_scales64(pages, length)
        j = np.arange(length)
        shown = ~np.isin(j // pool.T, hidden_pages)
        pos = (length - n + np.arange(n))[:, None]
        see = np.broadcast_to(shown[None], (n, length)).copy()
        if causal:
            see &= j[None] <= pos
        if window:
            see &= j[None] > pos - window
        for h in range(Hq):
            x = q[cu[b]:cu[b + 1], h].astype(np.float64)
            k, v = np.where(shown[:, None], K[:, h // G], 0), np.where(shown[:, None], V[:, h // G], 0)
            s = np.where(see, scale * (x @ k.T), -np.inf)
            size = np.where(see, scale * (np.abs(x) @ np.abs(k).T), 0).max(1)
            m = s.max(1, keepdims=True)
            with np.errstate(invalid="ignore"):
                p = np.where(see, np.exp(s - m), 0)
            total = p.sum(1)
            some = total > 0
            p = p / np.where(some, total, 1)[:, None]
            rows = np.arange(cu[b], cu[b + 1])
            out[rows, h] = p @ v
            with np.errstate(divide="ignore"):
                lse[rows, h] = np.where(some, np.where(some, m[:, 0], 0) + np.log(np.where(some, total, 1)), -np.inf)
            d = score_error(size, D)
            off[rows, h] = (weight_error() + 2 * d)[:, None] * (p @ np.abs(v))
            vs = np.where(shown, S[:, h // G], 0)
            codes = np.abs(v) / np.where(vs > 0, vs, 1)[:, None]
            off[rows, h] += SMALLEST_WEIGHT * (p * vs).max(1)[:, None] * (see.astype(np.float64) @ codes)
            lse_off[rows, h] = d + 2.0 ** -22 * (1 + np.abs(np.where(some, lse[rows, h], 0)))
    return out, lse, off, lse_off


# The weights p_j * vs_j of V's codes are held in binary16 with the largest
# seen so far at 2^4 at least: below 2^-14 they are rounded to multiples of
# 2^-24, so off by at most 2^-25, which is 2^-29 of the largest, for each
# position.
SMALLEST_WEIGHT = 2.0 ** -29


def weight_error():
    """A weight enters the second product as a binary16 value: half a step,
    2^-11 of it.  Sums in binary32 and the exponential and reciprocal
    instructions (one step each) add less than 2^-18 over a few thousand terms."""
    return 2.0 ** -11 + 2.0 ** -18


def score_error(size, D):
    """How far a score may be off, in natural units: D products summed in
    binary32 (2^-24 of the sum of |q k| each step), and four binary32 roundings
    (scale products, the shift by the maximum) of a number at most 1.45 * size
    + 64 + 15 in the exponent of two."""
    return (D + 8) * 2.0 ** -24 * size + 4 * 2.0 ** -24 * (1.45 * size + 79) * math.log(2)


def tolerance(out, off, dtype):
    """`off`, and half a step of the output type (at least its smallest step)."""
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * half
    return off + half * (np.abs(out) + off) + tiny
