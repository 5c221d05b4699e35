"""Plain CPU oracle of the operators of a step of many tokens -- TEST INFRASTRUCTURE ONLY.

Normalisation with int8 output, the paged 4-bit cache (append, read,
attention) and the 8-bit product, in fp64 with exactly the roundings that the
definitions in include/tern.h state. Nothing here is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .decode import bf16_round

__all__ = ["bf16_value", "norm_quantize", "rotate", "quantize4", "block_bytes", "Cache", "attention", "gemm_i8"]

F32 = np.float32


def bf16_value(v: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16, as fp32."""
    return (bf16_round(np.asarray(v, F32)).astype(np.uint32) << 16).view(F32)


def norm_quantize(mode: str, x, r, gain, eps: float, r_bf16: bool = False):
    """(v after the first step, xq int8, xscale fp32) of rows x, r (fp32 arrays holding the inputs' values)."""
    x = np.asarray(x, F32)
    if mode == "add":
        v = (x + r).astype(F32)
        v = bf16_value(v) if r_bf16 else v
    elif mode == "relu2":
        g = np.maximum(x, F32(0))
        v = ((g * g).astype(F32) * r).astype(F32)
    else:
        v = x
    f = (1.0 / np.sqrt((v.astype(np.float64) ** 2).mean(1) + np.float64(F32(eps)))).astype(F32)
    y = ((v * f[:, None]).astype(F32) * np.asarray(gain, F32)).astype(F32)
    a = np.abs(y).max(1).astype(F32)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.where(a > 0, F32(127) / a, F32(0)).astype(F32)
        w = (y * inv[:, None]).astype(F32)
    w = np.where(y == 0, F32(0), w)
    return v, np.clip(np.rint(w), -127, 127).astype(np.int8), (a / F32(127)).astype(F32)


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray) -> np.ndarray:
    """rotate_half of x fp32 [tokens][heads][d] with cos, sin fp32 [tokens][d/2], every product and sum rounded."""
    h = x.shape[-1] // 2
    a, b, c, s = x[..., :h], x[..., h:], cos[:, None], sin[:, None]
    lo = ((a * c).astype(F32) - (b * s).astype(F32)).astype(F32)
    hi = ((b * c).astype(F32) + (a * s).astype(F32)).astype(F32)
    return np.concatenate([lo, hi], -1)


def quantize4(x: np.ndarray):
    """(codes uint8, scale fp16, min fp16) of fp32 heads x [..., d]."""
    lo, hi = x.min(-1).astype(F32), x.max(-1).astype(F32)
    m = lo.astype(np.float16)
    s = ((hi - lo).astype(F32) / F32(15)).astype(F32).astype(np.float16)
    s32 = s.astype(F32)
    with np.errstate(divide="ignore"):
        inv = np.where(s32 > 0, F32(1) / s32, F32(0)).astype(F32)
    c = (((x - m.astype(F32)[..., None]).astype(F32)) * inv[..., None]).astype(F32)
    return np.clip(np.rint(c), 0, 15).astype(np.uint8), s, m


def block_bytes(page: int, d: int) -> int:
    return page * (d + 8)


class Cache:
    """The pages as bytes [num_pages][kv_heads][block], with the documented layout written out one token at a time."""

    def __init__(self, raw: np.ndarray, kv_heads: int, d: int, page: int):
        self.raw = raw.reshape(-1, kv_heads, block_bytes(page, d))
        self.kvh, self.d, self.page = kv_heads, d, page

    def put(self, page_id: int, slot: int, head: int, which: int, codes, scale, mn):
        """which: 0 keys, 1 values."""
        b, half = self.raw[page_id, head], self.page * self.d // 2
        at = which * half + slot * self.d // 2
        b[at:at + self.d // 2] = codes[0::2] | (codes[1::2] << 4)
        at = 2 * half + slot * 8 + which * 4
        b[at:at + 4] = np.array([scale, mn], np.float16).view(np.uint8)

    def get(self, page_id: int, slot: int, head: int, which: int):
        """(codes, scale, min) of one token."""
        b, half = self.raw[page_id, head], self.page * self.d // 2
        at = which * half + slot * self.d // 2
        byte = b[at:at + self.d // 2]
        codes = np.empty(self.d, np.uint8)
        codes[0::2], codes[1::2] = byte & 15, byte >> 4
        at = 2 * half + slot * 8 + which * 4
        s, m = b[at:at + 4].copy().view(np.float16)
        return codes, s, m

    def parts(self, table_row, n: int, head: int, which: int):
        """codes [n][d], scales [n], mins [n] (fp64) of the first n positions."""
        c, s, m = np.empty((n, self.d)), np.empty(n), np.empty(n)
        for j in range(n):
            c[j], s[j], m[j] = self.get(int(table_row[j // self.page]), j % self.page, head, which)
        return c, s, m


def attention(cache: Cache, table, starts, lens, heads: int, scale: float, q: np.ndarray, expanded: bool = False):
    """Outputs fp64 [tokens][heads][d] and a bound on how far the kernel's may be from them.

    The bound adds up: the bf16 rounding of the output, half a step 2^-8 of its value; the fp16 rounding of each
    probability times value scale w = p s, which enters as w c + p (m + 7.5 s) - 7.5 w and so weighs the code's distance
    from 7.5: 2^-11 sum p s |c - 7.5|; and the fp32 accumulation, a few roundings of 2^-23 (the tensor cores may cut
    instead of round) of the sums of magnitudes |m| + s c + 15 s, here and in the scores, whose error d in the exponent
    changes every probability by d. Sequences of more than 48 query rows per kv head (with
    `expanded` all) are computed from keys and values rounded to fp16, half a step 2^-11 of each element, and
    probabilities rounded to fp16."""
    d, kvh = cache.d, cache.kvh
    g = heads // kvh
    out = np.zeros((q.shape[0], heads, d))
    tol = np.zeros_like(out)
    for s in range(len(lens)):
        n = int(starts[s + 1] - starts[s])
        if n == 0:
            continue
        ln = int(lens[s])
        for h in range(kvh):
            kc, ks, km = cache.parts(table[s], ln, h, 0)
            vc, vs, vm = cache.parts(table[s], ln, h, 1)
            k, v = km[:, None] + ks[:, None] * kc, vm[:, None] + vs[:, None] * vc
            for i in range(n):
                seen = ln - n + i + 1
                if seen <= 0:
                    continue
                for e in range(g):
                    qi = q[starts[s] + i, h * g + e].astype(np.float64)
                    sc = k[:seen] @ qi * scale
                    p = np.exp(sc - sc.max())
                    p /= p.sum()
                    o = p @ v[:seen]
                    out[starts[s] + i, h * g + e] = o
                    mag = abs(scale) * np.abs(qi).sum() * (15 * ks[:seen] + np.abs(km[:seen])).max()
                    err = 2.0 ** -20 * (mag + np.abs(sc).max() + 1)
                    if expanded or n * g > 48:
                        err += 2.0 ** -11 * abs(scale) * np.abs(qi).sum() * np.abs(k[:seen]).max()
                        tol[starts[s] + i, h * g + e] += 1.01 * 2.0 ** -10 * (p @ np.abs(v[:seen]))
                    terms = p @ (np.abs(vm[:seen, None]) + vs[:seen, None] * (vc[:seen] + 15))
                    off = p @ (vs[:seen, None] * np.abs(vc[:seen] - 7.5))
                    tol[starts[s] + i, h * g + e] += (2.0 ** -8 * np.abs(o) + 1.01 * 2.0 ** -11 * off
                                                     + 2 * err * (p @ np.abs(v[:seen]) + np.abs(o)) + 2.0 ** -20 * terms)
    return out, tol


def gemm_i8(x: np.ndarray, sx: np.ndarray, w: np.ndarray, sw: np.ndarray) -> np.ndarray:
    """fl(fl(fl(acc) sw) sx) in fp32, acc the exact integer."""
    acc = x.astype(np.float64) @ w.astype(np.float64).T  # integers below 2^53: exact
    return ((acc.astype(F32) * sw[None]).astype(F32) * sx[:, None]).astype(F32)
