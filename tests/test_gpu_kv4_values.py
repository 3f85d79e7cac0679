"""kv4_attention of few rows where the values' scales lie far apart.

The bound is that of test_gpu_kv4_attention, with a weight's half step (2^-25,
where its product with the value's scale is an fp16 subnormal) held against the
largest such product of the same row and group: nothing that a row does not
see, or hardly sees, and nothing of another group may cost it precision."""
import numpy as np
import pytest
import torch

from tests import attention_ref as ref
from tests.test_gpu_kv4_attention import make, wlq

pytestmark = pytest.mark.gpu


def tight(q, cache, kv, table, scale, causal, window):
    """One sequence: (out, bound) in 64 bits with a weight's half step held against the row's and group's largest
    weight times value scale among the tokens it SEES, as the header states it for few rows."""
    n, Hq, D = q.shape
    P, hk, G = cache[0].shape[2], cache[0].shape[1], cache[3].shape[3]
    r = ref.attention(q, cache, np.array([0, n]), np.array([kv]), table, scale, causal, window)
    pages = table[0][: -(-kv // P)]
    k, v = ref.cache_values(cache[0], cache[1], pages, kv), ref.cache_values(cache[2], cache[3], pages, kv)
    vs = cache[3][torch.as_tensor(np.asarray(pages, dtype=np.int64), device=q.device)].double().transpose(0, 1).reshape(hk, -1, G)[:, :kv]
    i, j = torch.arange(n, device=q.device)[:, None] + (kv - n), torch.arange(kv, device=q.device)
    seen = (j <= i) & ((j > i - window) if window else True) if causal else torch.ones(n, kv, dtype=torch.bool, device=q.device)
    B = torch.empty(n, Hq, D, dtype=torch.float64, device=q.device)
    for h in range(Hq):
        g = h // (Hq // hk)
        p = torch.softmax(torch.where(seen, q[:, h].double() @ k[g].T * scale, float("-inf")), -1)
        top = (p[:, :, None] * vs[g]).amax(1).repeat_interleave(D // G, -1)               # [n, D]
        s = vs[g].repeat_interleave(D // G, -1)
        codes = torch.where(s > 0, v[g].abs() / torch.where(s > 0, s, 1.0), 0.0)
        B[:, h] = 2.0 ** -25 * top * (seen.double() @ codes)
    tol = 2.0 ** -8 * np.abs(r["out"]) + (r["A"] * (np.expm1(2 * r["E"]) + 2.0 ** -10 + 2.0 ** -16)[..., None] + B.cpu().numpy()) * (1 + 2.0 ** -8)
    return r["out"], tol


def check_tight(m, q, cache, cu, kv, table, causal=True, window=0, max_kv=None):
    dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (cu, kv, table)]
    got = ref.f64(m.kv4_attention(q, cache, *dev, q.shape[0], max_kv or int(kv[0]), causal=causal, window=window))
    want, tol = tight(q, cache, int(kv[0]), table, q.shape[2] ** -0.5, causal, window)
    err = np.abs(got - want)
    assert (err <= tol).all(), (np.nanmax(err / tol), np.linalg.norm(err) / np.linalg.norm(want))
    m.check_status()


def token(table, page, j):
    return int(table[0, j // page]), slice(None), j % page


FORMS = [(128, 32, 16), (128, 64, 64), (128, 128, 32), (64, 32, 32), (64, 64, 16)]


@pytest.mark.parametrize("D,group,page", FORMS)
@pytest.mark.parametrize("n,share", [(1, 1), (1, 8), (2, 8)])
@pytest.mark.parametrize("kv", [90, 1500, 9000])  # one part, parts joined by their cluster, parts joined by a second launch
def test_one_group_of_values_far_larger_than_the_others(D, group, page, n, share, kv):
    m = wlq()
    q, cache, cu, kvs, table = make(kv + share, [n], [kv], 2, share, D, group, page)
    if D > group:
        cache[3][..., 1] *= 2.0 ** 12
        cache[3][..., 0] *= 2.0 ** -8
    else:  # one token
        cache[3][token(table, page, kv // 3)] *= 2.0 ** 12
        cache[3][token(table, page, kv // 2)] *= 2.0 ** -8
    check_tight(m, q, cache, cu, kvs, table)


@pytest.mark.parametrize("D,group,page", FORMS)
@pytest.mark.parametrize("n,share", [(1, 1), (1, 8), (2, 8)])
@pytest.mark.parametrize("kv", [90, 1500, 9000])
def test_large_values_that_a_row_hardly_sees(D, group, page, n, share, kv):
    """One token with values 2^20 times the others': some rows see next to nothing of it, others nothing else."""
    m = wlq()
    q, cache, cu, kvs, table = make(kv + share + 1, [n], [kv], 1, share, D, group, page)
    cache[3].mul_(2.0 ** -7)
    at = token(table, page, kv // 3)
    cache[3][at] = 2.0 ** 12
    u = torch.where(torch.randn(D, generator=torch.Generator().manual_seed(3)) > 0, 1, -1)
    cache[0][at] = torch.from_numpy(ref.pack4((7 * u).numpy().astype(np.int8))).cuda()
    cache[1][at] = 0.5
    away = (u * 1.0).bfloat16().cuda()
    q[0, 0] = -away                     # a score of -3.5 sqrt(D): e^-28 or e^-40
    if q.shape[1] > 1:
        q[0, 1] = away                  # nothing else
        q[-1, 2] = -4 * away
    check_tight(m, q, cache, cu, kvs, table)


@pytest.mark.parametrize("D,group,page", FORMS)
@pytest.mark.parametrize("n,share", [(1, 4), (3, 8)])
@pytest.mark.parametrize("kv,window", [(90, 50), (1500, 1111), (9000, 8500)])
def test_large_values_behind_the_window(D, group, page, n, share, kv, window):
    """Values 2^20 times the others' in the token just before the first one that is seen, and in those before it."""
    m = wlq()
    q, cache, cu, kvs, table = make(kv + share + 2, [n], [kv], 2, share, D, group, page)
    cache[3].mul_(2.0 ** -7)
    for j in range(max(0, kv - n - window - 20), kv - n - window + 1):
        cache[3][token(table, page, j)] = 2.0 ** 12
    check_tight(m, q, cache, cu, kvs, table, window=window)


@pytest.mark.parametrize("D,group,page", FORMS)
def test_values_whose_products_fall_and_climb(D, group, page):
    """Weights and value scales that move by powers of two from token to token, against each other and together; long
    stretches of zero scales; a cache of zeros."""
    m = wlq()
    kv = 700
    for order in range(4):
        q, cache, cu, kvs, table = make(order + D, [1], [kv], 1, 8, D, group, page)
        q[:] = 1.0
        for j in range(kv):
            t = (j, kv - 1 - j, abs(j - kv // 2), j)[order] / kv
            cache[0][token(table, page, j)] = torch.from_numpy(ref.pack4(np.ones(D, dtype=np.int8))).cuda()
            cache[1][token(table, page, j)] = 8.0 * t               # scores up to 8 sqrt(D): 2^90 or 2^130
            e = (-20 * t, 10 * t, 12 - 24 * t, 0)[order]
            cache[3][token(table, page, j)] = 2.0 ** round(e) if order < 3 else (0.0 if 100 < j < 690 else 1.0)
        check_tight(m, q, cache, cu, kvs, table)
    q, cache, cu, kvs, table = make(5, [1], [kv], 1, 8, D, group, page)
    cache[3][torch.isfinite(cache[3])] = 0.0
    check_tight(m, q, cache, cu, kvs, table)
