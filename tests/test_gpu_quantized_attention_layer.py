"""The attention layer's operators together, as a model's layer calls them:
W8A8 projection of the hidden states, norm and rotation of the queries, the
append of keys and values into the 4-bit cache, attention over it, W8A8
output projection -- a first chunk of prompt, then single tokens, two
sequences of different lengths in one batch.

The reference is 64-bit throughout but for what the layer itself rounds: each
step's bf16 (or int8, 4-bit) result is taken from the 64-bit value of the
step.  Steps that round differently by one place move later ones a little, so
the layer's output is held to 2 % of its 2-norm (bf16 hands every step 2^-8 /
sqrt 3 = 0.23 %, int8 activations 1 / (127 sqrt 12) of the largest value's
step, about 0.9 %, at each of the two projections: 1.3 % in squares), and
every step on its own inputs to its own bound elsewhere."""
import numpy as np
import pytest
import torch

from tests import attention_ref as ref

pytestmark = pytest.mark.gpu


def wlq():
    import weight_only_quantized_rtn_b200 as m
    return m


def w8a8_64(x, wq, ws, b):
    xs = (np.abs(x).max(1) / 127).astype(np.float32).astype(np.float64)
    xq = np.rint(x / np.where(xs > 0, xs, 1)[:, None])
    return ref.bf16_rne((xq @ wq.T) * xs[:, None] * ws + b)


@pytest.mark.parametrize("group,sections,interleaved", [(32, (32,), False), (64, (12, 10, 10), True)])
def test_prompt_then_single_tokens(group, sections, interleaved):
    m = wlq()
    hidden, Hq, Hk, D, page, pages = 512, 8, 2, 64, 16, 24
    g = torch.Generator().manual_seed(group)
    Wqkv, Wo = torch.randn((Hq + 2 * Hk) * D, hidden, generator=g) * 0.06, torch.randn(hidden, Hq * D, generator=g) * 0.06
    bias = (torch.randn((Hq + 2 * Hk) * D, generator=g) * 0.1).bfloat16()
    qkv_q, qkv_s = m.quantize(Wqkv.cuda(), 8, 0)
    o_q, o_s = m.quantize(Wo.cuda(), 8, 0)
    wq = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16()
    wk = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16()
    pairs = sum(sections)
    freq = (100.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()
    cache = m.Kv4Cache(pages, Hk, page, D, group)
    table = torch.randperm(pages, generator=g)[:22].reshape(2, 11).to(torch.int32)
    keys = [np.zeros((0, Hk, D)), np.zeros((0, Hk, D))]   # the reference's cache: exact values as they were rounded
    vals = [np.zeros((0, Hk, D)), np.zeros((0, Hk, D))]
    lens = [0, 0]
    for q_lens in ([70, 37], [1, 1], [1, 1], [5, 0]):
        T = sum(q_lens)
        cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        lens = [a + b for a, b in zip(lens, q_lens)]
        x = torch.randn(T, hidden, generator=g).bfloat16()
        pos = np.concatenate([np.arange(n - q, n) for n, q in zip(lens, q_lens)])
        pos = np.stack([pos // (7 ** a) for a in range(len(sections))], 1).astype(np.int32)
        dev = [torch.from_numpy(a).cuda() for a in (cu, np.array(lens, dtype=np.int32))] + [table.cuda()]
        rope = dict(positions=torch.from_numpy(pos).cuda(), inv_freq=freq.cuda(), sections=sections, interleaved=interleaved)
        qkv = m.w8a8_linear(x.cuda(), qkv_q, qkv_s.reshape(-1), bias=bias.cuda()).view(T, Hq + 2 * Hk, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        m.kv4_append(cache, k, v, *dev, max(q_lens), k_weight=wk.cuda(), **rope)
        q = m.qk_norm_rope(q, None, q_weight=wq.cuda(), **rope)[0]
        o = m.kv4_attention(q, cache, *dev, max(q_lens), max(lens))
        y = m.w8a8_linear(o.view(T, Hq * D), o_q, o_s.reshape(-1), out_dtype=torch.float32)
        m.check_status()
        # the same in 64 bits
        r = w8a8_64(ref.f64(x), qkv_q.cpu().double().numpy(), ref.f64(qkv_s).reshape(-1), ref.f64(bias)).reshape(T, Hq + 2 * Hk, D)
        rq = ref.bf16_rne(ref.norm_rope(r[:, :Hq], ref.f64(wq), 1e-6, pos, freq.numpy(), sections, interleaved))
        rk = ref.key_bits(ref.norm_rope(r[:, Hq:Hq + Hk], ref.f64(wk), 1e-6, pos, freq.numpy(), sections, interleaved))
        ro = np.zeros((T, Hq, D))
        for b in range(2):
            rows = slice(cu[b], cu[b + 1])
            for store, new in ((keys, rk[rows]), (vals, r[rows, Hq + Hk:])):
                c, s = ref.quantize4(new, group)
                store[b] = np.concatenate([store[b], (c.reshape(*s.shape, group) * s[..., None]).reshape(new.shape)])
            n = q_lens[b]
            for h in range(Hq):
                z = rq[rows, h] @ keys[b][:, h // (Hq // Hk)].T / np.sqrt(D)
                z = np.where(np.arange(lens[b])[None] <= np.arange(n)[:, None] + lens[b] - n, z, -np.inf)
                e = np.exp(z - z.max(-1, keepdims=True)) if n else z
                ro[rows, h] = (e / e.sum(-1, keepdims=True)) @ vals[b][:, h // (Hq // Hk)] if n else 0
        ry = w8a8_64(ref.bf16_rne(ro).reshape(T, -1), o_q.cpu().double().numpy(), ref.f64(o_s).reshape(-1), 0.0)
        got = y.double().cpu().numpy()
        assert np.linalg.norm(got - ry) <= 0.02 * np.linalg.norm(ry)
