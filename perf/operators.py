"""Workloads of the quantized attention layer's operators: what is measured.

The operators are the steps around the quantized Linear of a transformer's attention layer:

- ``rope``    norms of queries and keys for each head and the rotary position (one to three axes), one pass
- ``append``  keys and values into a paged cache held in 4 bits, norm and rotation applied on the way
- ``attend``  attention over that cache: single tokens, chunks, causal prompts, sliding windows
- ``w8a8``    the Linear in 8-bit integers, a scale for each token and for each output channel

``run`` computes them in elementary torch operations where ``own`` is false and calls the library where it is true.
"""
import math
import random

import torch

own = False


def _api():
    import weight_only_quantized_rtn_b200 as wlq

    return wlq


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One decoding step of 16 streams: queries and keys right after the projections, where latency counts.
        dict(name="rope-step", op="rope", tokens=16, q_heads=32, k_heads=8, dim=128, rot=128, axes=1, interleaved=False, far=1 << 20),
        # Four latent frames of a video transformer's chunk (6240 tokens, hidden 4096): time, height and width positions.
        dict(name="rope-chunk", op="rope", tokens=6240, q_heads=32, k_heads=32, dim=128, rot=128, axes=3, interleaved=True, far=64),
        # One step of 33 streams appends one token each.
        dict(name="append-step", op="append", batch=33, q=1, kv=2049, k_heads=8, dim=128, group=64, page=16, rot=128, axes=1, interleaved=False, lens=1),
        # Four latent frames enter the cache of one stream.
        dict(name="append-chunk", op="append", batch=1, q=6240, kv=7800, k_heads=32, dim=128, group=128, page=64, rot=128, axes=3, interleaved=True, lens=2),
        # One stream, one token, a short context: the shortest call.
        dict(name="attend-one", op="attend", batch=1, q=1, kv=1560, q_heads=32, k_heads=8, dim=128, group=64, page=16, causal=True, window=0, lens=3),
        # A serving batch's decoding step, ragged contexts.
        dict(name="attend-batch", op="attend", batch=64, q=1, kv=8191, q_heads=32, k_heads=8, dim=128, group=64, page=32, causal=True, window=0, lens=4),
        # Two long contexts, one token each: little to share out, much to read.
        dict(name="attend-long", op="attend", batch=2, q=1, kv=131072, q_heads=64, k_heads=8, dim=128, group=32, page=128, causal=True, window=0, lens=5),
        # One latent frame (1560 tokens) looks at itself and four cached frames, every head its own keys.
        dict(name="attend-chunk", op="attend", batch=1, q=1560, kv=7800, q_heads=32, k_heads=32, dim=128, group=128, page=64, causal=False, window=0, lens=6),
        # Ragged prompts, causal, narrow heads.
        dict(name="attend-prompt", op="attend", batch=3, q=4097, kv=4097, q_heads=32, k_heads=8, dim=64, group=32, page=16, causal=True, window=0, lens=7),
        # Few tokens through an attention projection: the weight's bytes count.
        dict(name="w8a8-step", op="w8a8", tokens=16, n=4096, k=4096, bias=True),
        # One latent frame up to the hidden layer of the MLP.
        dict(name="w8a8-frame", op="w8a8", tokens=1560, n=16384, k=4096, bias=True),
        # Four latent frames back down.
        dict(name="w8a8-down", op="w8a8", tokens=6240, n=4096, k=16384, bias=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "w8a8"])
    dim = rng.choice([64, 128])
    axes = rng.choice([1, 2, 3])
    rot = rng.choice([dim, dim, dim // 2])
    k_heads = rng.choice([1, 2, 4, 8, 16, 32])
    page = rng.choice([16, 32, 64, 128])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    inter = rng.random() < 0.5
    if op == "rope":
        tokens = _log(rng, 1, 6240)
        q_heads = rng.choice([h for h in (8, 16, 32) if h >= k_heads] or [32])
        return dict(op=op, tokens=tokens, q_heads=q_heads, k_heads=k_heads, dim=dim, rot=rot, axes=axes, interleaved=inter, far=_log(rng, 16, 1 << 20))
    if op == "append":
        batch = _log(rng, 1, 64)
        q = 1 if rng.random() < 0.3 else _log(rng, 1, 6240 // batch)
        return dict(op=op, batch=batch, q=q, kv=q + _log(rng, 1, 2048), k_heads=k_heads, dim=dim, group=group, page=page, rot=rot, axes=axes,
                    interleaved=inter, lens=rng.randrange(1 << 20))
    if op == "attend":
        share = rng.choice([1, 2, 4, 8])
        while k_heads * share > 64:
            share //= 2
        q_heads = k_heads * share
        if rng.random() < 0.5:  # single tokens
            batch = _log(rng, 1, 64)
            q, kv = 1, _log(rng, 1, min(65536, (1 << 22) // (batch * k_heads)))
        else:
            q = _log(rng, 2, 4096)
            batch = _log(rng, 1, max(1, min(8, 4096 // q)))
            kv = q + _log(rng, 1, 4096)
            while batch * q_heads * q * kv > 350_000_000 and q_heads > 1:
                q_heads = max(1, q_heads // 2)
                k_heads = min(k_heads, q_heads)
        causal = rng.random() < 0.6
        window = _log(rng, 16, 4096) if causal and rng.random() < 0.4 else 0
        return dict(op=op, batch=batch, q=q, kv=kv, q_heads=q_heads, k_heads=k_heads, dim=dim, group=group, page=page, causal=causal, window=window,
                    lens=rng.randrange(1 << 20))
    return dict(op=op, tokens=_log(rng, 1, 6240), n=8 * _log(rng, 32, 1024), k=16 * _log(rng, 16, 512), bias=rng.random() < 0.7)


def _lens(c):
    """Tokens of this call and tokens in the cache after it, for each sequence: the first has the most, the others are spread below."""
    r = random.Random(c["lens"])
    q_lens, kv_lens = [], []
    for b in range(c["batch"]):
        f = 1.0 if b == 0 else r.uniform(0.3, 1.0)
        kv = max(1, int(c["kv"] * f))
        q = c["q"] if b == 0 else max(1, int(c["q"] * r.uniform(0.3, 1.0)))
        q_lens.append(min(q, kv))
        kv_lens.append(kv)
    return q_lens, kv_lens


def _sections(c):
    """Rotated pairs of each axis, the first axis with what is left over."""
    pairs, a = c["rot"] // 2, c["axes"]
    return (pairs - (a - 1) * (pairs // a),) + (pairs // a,) * (a - 1)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rope_inputs(c, g, tokens, first):
    """Frequencies of each axis' pairs and the positions: consecutive tokens from `first`, or (time, height, width) of a 30 x 52 frame's tokens."""
    freqs = []
    for n in _sections(c):
        freqs.append(torch.pow(torch.tensor(10000.0, dtype=torch.float64), -torch.arange(n, dtype=torch.float64) / n).float())
    t = torch.arange(tokens, device="cuda")
    if c["axes"] == 1:
        pos = (first + t)[:, None]
    elif c["axes"] == 2:
        pos = torch.stack([first + t // 52, t % 52], 1)
    else:
        pos = torch.stack([first + t // 1560, t // 52 % 30, t % 52], 1)
    return dict(positions=pos.to(torch.int32).contiguous(), inv_freq=torch.cat(freqs).cuda(), sections=_sections(c), interleaved=c["interleaved"])


def _pack_words(q):
    """Codes -7..7 [..., D] as the cache's bytes [..., D / 2]: words of 8 codes, code t of a word at nibble t / 2 (even t) or 4 + t / 2 (odd t)."""
    u = (q + 8).to(torch.uint8).reshape(*q.shape[:-1], -1, 8)
    lo, hi = u[..., 0::2], u[..., 1::2]  # nibbles 0..3 and 4..7
    b = torch.stack([lo[..., 0] | lo[..., 1] << 4, lo[..., 2] | lo[..., 3] << 4, hi[..., 0] | hi[..., 1] << 4, hi[..., 2] | hi[..., 3] << 4], -1)
    return b.reshape(*q.shape[:-1], -1).contiguous()


def _unpack_words(b):
    """The inverse of _pack_words, as int32 codes -7..7 (8 below the stored values)."""
    b = b.reshape(*b.shape[:-1], -1, 4).to(torch.int32)
    n = torch.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], 8)  # nibbles 0..7
    t = torch.stack([n[..., :4], n[..., 4:]], -1)                    # code 2 j at nibble j, 2 j + 1 at nibble 4 + j
    return t.reshape(*b.shape[:-2], -1) - 8


def _cache(c, g, pages, spread):
    """A filled cache: values of a normal distribution, for the keys some channels larger, quantized to 4 bits."""
    out = []
    for s in spread:
        x = _randn(g, pages, c["k_heads"], c["page"], c["dim"]) * s
        x = x.reshape(pages, c["k_heads"], c["page"], c["dim"] // c["group"], c["group"])
        sc = (x.abs().amax(-1) / 7).half()
        q = torch.round(x / sc.float()[..., None]).clamp_(-7, 7).to(torch.int32)
        out += [_pack_words(q.reshape(pages, c["k_heads"], c["page"], c["dim"])), sc.contiguous()]
        del x, q
    return tuple(out)


def _table(c, g, kv_lens):
    """Each sequence's pages, scattered over the pool."""
    per = -(-max(kv_lens) // c["page"])
    pages = len(kv_lens) * per + 3
    perm = torch.randperm(pages, generator=g, device="cuda")[: len(kv_lens) * per]
    return perm.to(torch.int32).reshape(len(kv_lens), per).contiguous(), pages


def _cu(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    s = dict(case=c)
    if op == "w8a8":
        w = _randn(g, c["n"], c["k"]) * 0.02
        ws = w.abs().amax(1) / 127
        s["wq"] = torch.round(w / ws[:, None]).clamp_(-127, 127).to(torch.int8)
        s["ws"] = ws.contiguous()
        s["x"] = _randn(g, c["tokens"], c["k"]).bfloat16()
        s["bias"] = (_randn(g, c["n"]) * 0.01).bfloat16() if c["bias"] else None
        return s
    dim = c["dim"]
    spread = 1.0 + 3.0 * (torch.rand(dim, generator=g, device="cuda") > 0.95)
    if op == "rope":
        t = c["tokens"]
        # views of one fused projection output, as the Linear leaves them
        qkv = (_randn(g, t, c["q_heads"] + 2 * c["k_heads"], dim) * spread).bfloat16()
        s["q"], s["k"] = qkv[:, : c["q_heads"]], qkv[:, c["q_heads"] : c["q_heads"] + c["k_heads"]]
        s["q_weight"] = (1 + 0.2 * _randn(g, dim)).bfloat16()
        s["k_weight"] = (1 + 0.2 * _randn(g, dim)).bfloat16()
        s.update(_rope_inputs(c, g, t, c["far"]))
        return s
    q_lens, kv_lens = _lens(c)
    total = sum(q_lens)
    s["table"], pages = _table(c, g, kv_lens)
    s["cu"], s["kv"] = _cu(q_lens), torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    s["max_q"], s["max_kv"], s["total"] = max(q_lens), max(kv_lens), total
    if op == "append":
        kv = (_randn(g, total, 2 * c["k_heads"], dim) * spread).bfloat16()
        s["k"], s["v"] = kv[:, : c["k_heads"]], kv[:, c["k_heads"] :]
        s["k_weight"] = (1 + 0.2 * _randn(g, dim)).bfloat16()
        s.update(_rope_inputs(c, g, total, kv_lens[0] - q_lens[0]))
        h, p = c["k_heads"], c["page"]
        s["cache"] = tuple(torch.zeros(pages, h, p, n, dtype=t, device="cuda") for n, t in
                           ((dim // 2, torch.uint8), (dim // c["group"], torch.float16)) * 2)
        return s
    s["cache"] = _cache(c, g, pages, (spread, torch.ones((), device="cuda")))
    s["q"] = _randn(g, total, c["q_heads"], dim).bfloat16()
    return s


# ------------------------------------------------------------------ the plain forms
def _angles(s):
    """cos and sin [T, 1, rot / 2] in 64 bits: far positions need them."""
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"), torch.tensor(s["sections"], device="cuda"),
                                   output_size=sum(s["sections"]))
    a = s["positions"].double()[:, axis] * s["inv_freq"].double()
    return a.cos()[:, None], a.sin()[:, None]


def _plain_norm_rope(x, weight, cos, sin, interleaved, eps=1e-6):
    """x [T, H, D] normed by its root mean square over D and rotated, in cos' type, rounded once to bf16."""
    x = x.to(cos.dtype)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.to(cos.dtype)
    rot = 2 * cos.shape[-1]
    y = x[..., :rot]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y.chunk(2, -1)
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def _plain_quantized(x, group):
    """bf16 x as the values its 4-bit form stands for, rounded to bf16: scales fp16(max / 7), codes to the nearest, ties to even (64 bits: next to a border)."""
    x = x.double().reshape(*x.shape[:-1], -1, group)
    sc = (x.abs().amax(-1, keepdim=True) / 7).half().double()
    q = torch.where(sc > 0, torch.round(x / torch.where(sc > 0, sc, 1.0)).clamp(-7, 7), 0.0)
    return (q * sc).flatten(-2).to(torch.bfloat16)


def _plain_values(codes, scales):
    """[..., D / 2] bytes and [..., D / group] scales as fp32 values [..., D]."""
    q = _unpack_words(codes).float()
    return (q.reshape(*scales.shape, -1) * scales.float()[..., None]).flatten(-2)


def _plain_attend(s):
    c = s["case"]
    kc, ks, vc, vs = s["cache"]
    table, cu, kv_lens = s["table"].long(), s["cu"].long(), s["kv"].long()
    batch, hk, dim = c["batch"], c["k_heads"], c["dim"]
    share = c["q_heads"] // hk
    n, m = table.shape[1] * c["page"], s["max_q"]
    k = _plain_values(kc[table], ks[table]).transpose(1, 2).reshape(batch, hk, n, dim)
    v = _plain_values(vc[table], vs[table]).transpose(1, 2).reshape(batch, hk, n, dim)
    q_lens = cu[1:] - cu[:-1]
    i = torch.arange(m, device="cuda")
    rows = (cu[:-1, None] + torch.minimum(i, (q_lens - 1).clamp(min=0)[:, None])).clamp(max=s["total"] - 1)
    q = s["q"].float()[rows].reshape(batch, m, hk, share, dim).permute(0, 2, 3, 1, 4).reshape(batch, hk, share * m, dim)
    z = (q @ k.transpose(-1, -2)).reshape(batch, hk, share, m, n) * (dim ** -0.5)
    at = (kv_lens - q_lens)[:, None] + i                                # position of query i
    j = torch.arange(n, device="cuda")
    seen = (j < kv_lens[:, None])[:, None].expand(batch, m, n)
    if c["causal"]:
        seen = seen & (j <= at[..., None])
        if c["window"]:
            seen = seen & (j > at[..., None] - c["window"])
    z = z.masked_fill(~seen[:, None, None], float("-inf"))
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top > float("-inf"), top, 0.0))
    total = e.sum(-1, keepdim=True)
    o = (e.reshape(batch, hk, share * m, n) @ v).reshape(batch, hk, share, m, dim) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, m, hk * share, dim)
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o[b, t - cu[b]].to(torch.bfloat16)


def _plain_w8a8(s):
    x = s["x"].double()
    xs = (x.abs().amax(1, keepdim=True) / 127).float().double()
    xq = torch.where(xs > 0, torch.round(x / torch.where(xs > 0, xs, 1.0)).clamp(-127, 127), 0.0).float()
    y = (xq @ s["wq"].float().t()) * (xs.float() * s["ws"])
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        wlq = _api()
        if op == "w8a8":
            return wlq.w8a8_linear(s["x"], s["wq"], s["ws"], bias=s["bias"])
        if op == "rope":
            return wlq.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["sections"], s["interleaved"],
                                    q_weight=s["q_weight"], k_weight=s["k_weight"])
        if op == "append":
            wlq.kv4_append(s["cache"], s["k"], s["v"], s["cu"], s["kv"], s["table"], s["max_q"], s["positions"], s["inv_freq"], s["sections"],
                           s["interleaved"], k_weight=s["k_weight"])
            return wlq.kv4_read(s["cache"], s["cu"], s["kv"], s["table"], s["max_q"], s["total"])
        return wlq.kv4_attention(s["q"], s["cache"], s["cu"], s["kv"], s["table"], s["max_q"], s["max_kv"], causal=c["causal"], window=c["window"])
    if op == "w8a8":
        return _plain_w8a8(s)
    if op == "attend":
        return _plain_attend(s)
    cos, sin = _angles(s)
    if op == "append":  # in 64 bits up to the codes: a key next to a border would fall on its other side
        k = _plain_norm_rope(s["k"], s["k_weight"], cos, sin, s["interleaved"])
        return _plain_quantized(k, c["group"]), _plain_quantized(s["v"], c["group"])
    cos, sin = cos.float(), sin.float()
    return (_plain_norm_rope(s["q"], s["q_weight"], cos, sin, s["interleaved"]), _plain_norm_rope(s["k"], s["k_weight"], cos, sin, s["interleaved"]))


def work(case):
    """Bytes: each input once (of the cache, what the masks leave visible to some query), each output once. Flops: products and sums of the definition."""
    c = case
    op = c["op"]
    if op == "w8a8":
        m, n, k = c["tokens"], c["n"], c["k"]
        return dict(bytes=2 * m * k + n * k + 4 * n + 2 * m * n + (2 * n if c["bias"] else 0), flops=2 * m * n * k)
    dim = c["dim"]
    if op == "rope":
        v = c["tokens"] * (c["q_heads"] + c["k_heads"]) * dim
        return dict(bytes=4 * v + 4 * c["tokens"] * c["axes"] + 2 * c["rot"] + 4 * dim, flops=8 * v)
    q_lens, kv_lens = _lens(c)
    total = sum(q_lens)
    row = dim // 2 + 2 * (dim // c["group"])
    if op == "append":  # the rows in, the cache's rows out, and both as values again
        v = 2 * total * c["k_heads"]
        return dict(bytes=v * (2 * dim + row) + v * (row + 2 * dim) + 4 * total * c["axes"] + 2 * c["rot"] + 2 * dim, flops=16 * v * dim)
    pairs = keys = 0
    for q, kv in zip(q_lens, kv_lens):
        if not c["causal"]:
            pairs, keys = pairs + q * kv, keys + kv
            continue
        w = c["window"] or kv
        keys += kv - max(0, kv - q + 1 - w)
        first = kv - q
        ramp = max(0, min(kv, w - 1) - first)  # queries whose window starts before the sequence
        pairs += min(w, kv) * (q - ramp) + ramp * first + ramp * (ramp + 1) // 2
    return dict(bytes=2 * keys * c["k_heads"] * row + 4 * total * c["q_heads"] * dim, flops=4 * pairs * c["q_heads"] * dim)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_normed(x, weight, s):
    """Each head's vector over its root mean square, times the weight; then each pair (a, b) as the complex number a + i b times e^(i angle)."""
    x = x.double()
    n = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1]
    x = x / torch.sqrt(n + 1e-6) * weight.double()
    angle, first = [], 0
    for a, count in enumerate(s["sections"]):
        angle.append(s["positions"][:, a : a + 1].double() * s["inv_freq"][first : first + count].double())
        first += count
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.cat(angle, 1))[:, None]
    if s["interleaved"]:
        re, im = torch.arange(0, 2 * first, 2, device="cuda"), torch.arange(1, 2 * first, 2, device="cuda")
    else:
        re, im = torch.arange(first, device="cuda"), torch.arange(first, 2 * first, device="cuda")
    z = torch.complex(x[..., re], x[..., im]) * turn
    x[..., re], x[..., im] = z.real, z.imag
    return x


def _exact_rounded(x, group):
    """x [..., D] in 64 bits to the nearest 4-bit values: bf16, then steps of fp16(max / 7)."""
    x = x.to(torch.bfloat16).double()
    out = torch.zeros_like(x)
    for first in range(0, x.shape[-1], group):
        part = x[..., first : first + group]
        step = (part.abs().max(-1, keepdim=True).values / 7).to(torch.float16).double()
        out[..., first : first + group] = torch.nan_to_num(torch.round(part / step)).clamp(-7, 7) * step
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    op = c["op"]
    if op == "rope":
        return _exact_normed(s["q"], s["q_weight"], s), _exact_normed(s["k"], s["k_weight"], s)
    if op == "append":
        return _exact_rounded(_exact_normed(s["k"], s["k_weight"], s), c["group"]), _exact_rounded(s["v"], c["group"])
    if op == "w8a8":
        x = s["x"].double()
        step = (x.abs().max(1).values / 127).to(torch.float32).double()
        codes = torch.nan_to_num(torch.round(x / step[:, None])).clamp(-127, 127)
        y = torch.einsum("mk,nk->mn", codes, s["wq"].double()) * step[:, None] * s["ws"].double()
        return y if s["bias"] is None else y + s["bias"].double()
    q_lens, kv_lens = _lens(c)
    kc, ks, vc, vs = s["cache"]
    share, dim, page = c["q_heads"] // c["k_heads"], c["dim"], c["page"]
    out = torch.zeros(s["total"], c["q_heads"], dim, dtype=torch.float64, device="cuda")
    first = 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        used = s["table"][b, : -(-n // page)].long()
        i, j = torch.arange(m, device="cuda")[:, None] + (n - m), torch.arange(n, device="cuda")
        seen = torch.ones(m, n, dtype=torch.bool, device="cuda")
        if c["causal"]:
            seen = j <= i
            if c["window"]:
                seen &= j > i - c["window"]
        for h in range(c["k_heads"]):
            k, v = ((_unpack_words(codes[used, h]).double().reshape(-1, dim // c["group"], c["group"]) *
                     scales[used, h].double().reshape(-1, dim // c["group"], 1)).reshape(-1, dim)[:n] for codes, scales in ((kc, ks), (vc, vs)))
            for a in range(h * share, (h + 1) * share):
                z = torch.where(seen, s["q"][first : first + m, a].double() @ k.T / math.sqrt(dim), float("-inf"))
                out[first : first + m, a] = torch.softmax(z, -1) @ v
        first += m
    return out
