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


def key_bits(y: np.ndarray) -> np.ndarray:
    """Real keys as the cache rounds them before their codes: to fp32, from there to bf16 (as fp64 values)."""
    return bf16_rne(np.asarray(y).astype(np.float32).astype(np.float64))


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
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
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
    words = np.ascontiguousarray(b).view(np.uint32).reshape(*b.shape[:-1], D // 8, 1)
    t = np.arange(8)
    nib = np.where(t % 2 == 0, t // 2, 4 + t // 2)
    return (((words >> (4 * nib).astype(np.uint32)) & 15).astype(np.int8) - 8).reshape(*b.shape[:-1], D)


def cache_values(codes, scales, pages, n):
    """The first n cached tokens' values [heads, n, D] (fp64, the tensors' device) on the given pages; NaN on pages out of range."""
    P, half, G = codes.shape[2], codes.shape[3], scales.shape[3]
    H, D = codes.shape[1], 2 * half
    pages = torch.as_tensor(np.asarray(pages, dtype=np.int64), device=codes.device)
    ok = (pages >= 0) & (pages < codes.shape[0])
    at = torch.where(ok, pages, torch.zeros_like(pages))
    c, s = codes[at], scales[at].double()
    shift = torch.tensor([4 * (t // 2 if t % 2 == 0 else 4 + t // 2) for t in range(8)], device=codes.device)
    w = c.contiguous().view(torch.int32).long() & 0xFFFFFFFF
    q = ((w[..., None] >> shift) & 15).double() - 8
    v = (q.reshape(len(pages), H, P, G, D // G) * s[..., None]).reshape(len(pages), H, P, D)
    v[~ok] = float("nan")
    return v.transpose(0, 1).reshape(H, -1, D)[:, :n]


def attention(q, cache, cu, kv_lens, table, scale, causal, window):
    """The 64-bit attention and what its error bounds need: a dict of fp64 arrays
    out, lse, E (the largest score error of fp16 keys), A (sum_j p_j |v_j|), B
    (2^-25 sum_j |q_j| max_j s_j, q and s the values' codes and scales).  Rows of no sequence are NaN; a query that sees
    nothing has out 0 and lse -inf."""
    T, Hq, D = q.shape
    dev = cache[0].device
    r = {k: torch.full((T, Hq) + ((D,) if k in ("out", "A", "B") else ()), float("nan"), dtype=torch.float64, device=dev)
         for k in ("out", "lse", "E", "A", "B")}
    q = q.double()
    P, hk = cache[0].shape[2], cache[0].shape[1]
    share = Hq // hk
    for b in range(len(kv_lens)):
        n, kv = int(cu[b + 1] - cu[b]), int(kv_lens[b])
        if n == 0:
            continue
        rows, pages = slice(int(cu[b]), int(cu[b + 1])), table[b][: -(-kv // P)]
        k, v = cache_values(cache[0], cache[1], pages, kv), cache_values(cache[2], cache[3], pages, kv)
        there = ~torch.isnan(k[0, :, 0])
        n_pages = torch.as_tensor(np.clip(np.asarray(pages, dtype=np.int64), 0, cache[0].shape[0] - 1), device=dev)
        vs = cache[3][n_pages].double().transpose(0, 1).reshape(hk, -1, cache[3].shape[3])[:, :kv]  # [heads, kv, groups]
        vs = torch.where(there[:, None], vs, 0.0).repeat_interleave(D // cache[3].shape[3], -1)
        vq = torch.where(vs > 0, v.nan_to_num() / torch.where(vs > 0, vs, 1.0), 0.0)
        b25 = 2.0 ** -25 * (vq.abs() * vs.amax((1, 2), keepdim=True)).sum(1)                           # [heads, D]
        k, v = torch.where(there[:, None], k, 0.0), torch.where(there[:, None], v, 0.0)
        i, j = torch.arange(n, device=dev)[:, None] + (kv - n), torch.arange(kv, device=dev)
        seen = torch.ones(n, kv, dtype=torch.bool, device=dev)
        if causal:
            seen = j <= i
            if window:
                seen = seen & (j > i - window)
        seen = seen & there
        for h in range(Hq):
            kh, vh = k[h // share], v[h // share]
            z = torch.where(seen, q[rows, h] @ kh.T * scale, float("-inf"))
            top = z.amax(-1, keepdim=True)
            top = torch.where(torch.isinf(top), 0.0, top)
            e = torch.exp(z - top)
            l = e.sum(-1, keepdim=True)
            p = e / torch.where(l > 0, l, 1.0)
            r["out"][rows, h], r["A"][rows, h] = p @ vh, p @ vh.abs()
            r["lse"][rows, h] = (torch.log(l) + top)[:, 0]
            r["E"][rows, h] = (q[rows, h].abs() @ kh.abs().T).amax(-1) * abs(scale) * (2.0 ** -11 + 2.0 ** -20)
            r["B"][rows, h] = b25[h // share]
    return {k: x.cpu().numpy() for k, x in r.items()}
