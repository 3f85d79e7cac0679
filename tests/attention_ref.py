"""Plain 64-bit forms of the attention layer's operators, for the tests: written
from the definitions in include/wlq.h with numpy, sharing nothing with the
CUDA code.  bf16 and fp16 values are handled as their exact fp64 values."""
from __future__ import annotations

import numpy as np
import torch


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def bf16_rne(x: np.ndarray) -> np.ndarray:
    """fp64 -> the nearest bf16 value (ties to even), as fp64, by integer steps on a scaled significand."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)                      # |m| in [1/2, 1)
    e = np.maximum(e, -125)                 # subnormals: a fixed last place
    step = np.ldexp(1.0, e - 8)
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(x), np.rint(x / step) * step, x)


def norm_rope(x, weight, eps, positions, inv_freq, sections, interleaved):
    """x [T, H, D] fp64 -> the real-number result in fp64 (not rounded)."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    if positions is None:
        return x
    T = x.shape[0]
    pos = np.asarray(positions, dtype=np.float64).reshape(T, -1)
    pairs = len(inv_freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    ang = pos[:, axis] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    ia, ib = (np.arange(0, 2 * pairs, 2), np.arange(1, 2 * pairs, 2)) if interleaved else (
        np.arange(pairs), np.arange(pairs, 2 * pairs))
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia], x[..., ib] = a * c - b * s, a * s + b * c
    return x


def quantize4(x, group):
    """fp64 values of bf16 x [..., D] -> (codes, fp16 scales as fp64 [..., D / group])."""
    g = x.reshape(*x.shape[:-1], -1, group)
    s = (np.abs(g).max(-1) / 7).astype(np.float16).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[..., None] > 0, np.clip(np.rint(g / s[..., None]), -7, 7), 0.0)
    return q.reshape(x.shape).astype(np.int8), s


def pack4(q):
    """codes [..., D] -> bytes [..., D / 2] by writing each nibble to its place."""
    D = q.shape[-1]
    words = np.zeros((*q.shape[:-1], D // 8), dtype=np.uint32)
    for d in range(D):
        t = d % 8
        nib = t // 2 if t % 2 == 0 else 4 + t // 2
        words[..., d // 8] |= (q[..., d].astype(np.int64) + 8).astype(np.uint32) << np.uint32(4 * nib)
    return words.view(np.uint8).reshape(*q.shape[:-1], D // 2)


def unpack4(b, D):
    words = np.ascontiguousarray(b).view(np.uint32).reshape(*b.shape[:-1], D // 8)
    q = np.zeros((*b.shape[:-1], D), dtype=np.int8)
    for d in range(D):
        t = d % 8
        nib = t // 2 if t % 2 == 0 else 4 + t // 2
        q[..., d] = ((words[..., d // 8] >> np.uint32(4 * nib)) & 15).astype(np.int8) - 8
    return q


def cache_values(cache, which, pages, head, n):
    """The first n tokens' values [n, D] (fp64) of one head on the given pages (-1 pages give NaN rows)."""
    codes, scales = (cache[0], cache[1]) if which == "k" else (cache[2], cache[3])
    P, D, G = codes.shape[2], codes.shape[3] * 2, scales.shape[3]
    out = np.full((len(pages) * P, D), np.nan)
    for i, p in enumerate(pages):
        if 0 <= p < codes.shape[0]:
            q = unpack4(codes[p, head].cpu().numpy(), D).astype(np.float64)
            s = f64(scales[p, head])
            out[i * P:(i + 1) * P] = (q.reshape(P, G, -1) * s[..., None]).reshape(P, D)
    return out[:n]


def attention(q, cache, cu, kv_lens, table, kv_heads, scale, causal, window):
    """(out [T, Hq, D], lse [T, Hq]) in fp64; rows of no sequence are NaN; a query that sees nothing has 0, -inf."""
    T, Hq, D = q.shape
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    share = Hq // kv_heads
    P = cache[0].shape[2]
    for b in range(len(kv_lens)):
        n, kv = cu[b + 1] - cu[b], kv_lens[b]
        pages = table[b][: -(-kv // P)]
        i, j = np.arange(n)[:, None] + (kv - n), np.arange(kv)[None]
        seen = np.ones((n, kv), dtype=bool)
        if causal:
            seen = j <= i
            if window:
                seen = seen & (j > i - window)
        for h in range(kv_heads):
            if kv:
                k, v = cache_values(cache, "k", pages, h, kv), cache_values(cache, "v", pages, h, kv)
                there = ~np.isnan(k[:, 0])
                k, v = np.nan_to_num(k), np.nan_to_num(v)
            else:
                k = v = np.zeros((0, D))
                there = np.zeros(0, dtype=bool)
            for g in range(share):
                z = q[cu[b]:cu[b + 1], h * share + g] @ k.T * scale
                z = np.where(seen & there, z, -np.inf)
                top = z.max(-1, initial=-np.inf, keepdims=True)
                e = np.exp(z - np.where(np.isfinite(top), top, 0.0))
                l = e.sum(-1)
                rows = slice(cu[b], cu[b + 1])
                out[rows, h * share + g] = (e @ v) / np.where(l > 0, l, 1.0)[:, None]
                with np.errstate(divide="ignore"):
                    lse[rows, h * share + g] = np.where(l > 0, np.log(l), -np.inf) + np.where(np.isfinite(top[:, 0]), top[:, 0], 0.0)
    return out, lse
