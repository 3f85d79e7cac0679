"""qk_norm_rope, kv4_append and kv4_read against 64-bit forms.

qk_norm_rope evaluates in fp32, within E = 9 * 2^-24 r (|a| + |b|) of the real
value y, and rounds once to bf16: the result lies between the bf16 values
nearest to y - E and y + E, which is what is checked; nearly all equal the one
nearest to y.  The cache promises the exact 4-bit rounding of the real keys
rounded to fp32 and then to bf16, so its codes are compared for equality: the
64-bit form is off by about 2^-49, and a border lies that close to a value
with a chance of about 2^-40."""
import numpy as np
import pytest
import torch

from tests import attention_ref as ref

pytestmark = pytest.mark.gpu


def wlq():
    import weight_only_quantized_rtn_b200 as m
    return m


def _rows(seed, T, H, D, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(spread * torch.randn(T, H, 1, generator=g))
    return x.bfloat16()


def _check_rows(got, x, weight, eps, positions, inv_freq, sections, interleaved):
    """got against the 64-bit rows, between the roundings of y - E and y + E."""
    y = ref.norm_rope(x, weight, eps, positions, inv_freq, sections, interleaved)
    n = ref.norm_rope(x, weight, eps, None, None, None, True)  # the pairs' inputs a, b (times r)
    size = np.abs(n)
    if positions is not None:
        pairs = len(inv_freq)
        ia, ib = (np.arange(0, 2 * pairs, 2), np.arange(1, 2 * pairs, 2)) if interleaved else (np.arange(pairs), np.arange(pairs, 2 * pairs))
        both = size[..., ia] + size[..., ib]
        size[..., ia], size[..., ib] = both, both
    E = 9 * 2.0 ** -24 * size
    assert ((ref.bf16_rne(y - E) <= got) & (got <= ref.bf16_rne(y + E))).all()
    assert (got == ref.bf16_rne(y)).mean() > 0.998  # E is 2^-12 of a bf16 step's half or less, but for differences of nearly equal products


def _freq(sections):
    return torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in sections]).float()


def _positions(seed, T, axes, far):
    g = np.random.default_rng(seed)
    p = g.integers(0, far, (T, axes))
    p[0] = 0
    if T > 1:
        p[1] = far - 1
    if T > 2:
        p[2] = -far // 2
    return torch.from_numpy(p.astype(np.int32))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,rot,sections,far", [
    (1, 1, 0, 64, (32,), 3),
    (1, 0, 3, 16, (8,), 1 << 20),
    (7, 5, 2, 48, (10, 14), 1 << 17),
    (33, 32, 8, 64, (12, 0, 20), 1 << 20),
    (260, 4, 1, 32, (3, 5, 7, 1), 1 << 28),
])
def test_norm_rope(D, interleaved, T, hq, hk, rot, sections, far):
    m = wlq()
    qkv = _rows(T + D, T, hq + 2 * hk, D).cuda()
    q, k = (qkv[:, :hq] if hq else None), (qkv[:, hq:hq + hk] if hk else None)
    g = torch.Generator().manual_seed(5)
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16(), (1 + 0.3 * torch.randn(D, generator=g)).bfloat16()
    pos, freq = _positions(T, T, len(sections), far), _freq(sections)
    qo, ko = m.qk_norm_rope(q, k, pos.cuda(), freq.cuda(), sections, interleaved, q_weight=wq.cuda(), k_weight=wk.cuda())
    for x, w, o in ((q, wq, qo), (k, wk, ko)):
        if x is None:
            assert o is None
            continue
        _check_rows(ref.f64(o), ref.f64(x), ref.f64(w), 1e-6, pos.numpy(), freq.numpy(), sections, interleaved)
    m.check_status()


@pytest.mark.parametrize("D", [64, 128])
def test_norm_only_rotation_only_neither_and_in_place(D):
    m = wlq()
    x = _rows(3, 21, 6, D).cuda()
    w = _rows(4, 1, 1, D, 0.0).reshape(D).cuda()
    pos, freq = _positions(1, 21, 1, 1000), _freq((D // 2,))
    o, none = m.qk_norm_rope(x, None, q_weight=w, eps=1e-5)
    assert none is None
    _check_rows(ref.f64(o), ref.f64(x), ref.f64(w), 1e-5, None, None, None, True)
    for inter in (False, True):
        o, _ = m.qk_norm_rope(x, None, pos[:, 0].contiguous().cuda(), freq.cuda(), interleaved=inter)
        _check_rows(ref.f64(o), ref.f64(x), None, 0.0, pos[:, 0].numpy(), freq.numpy(), (D // 2,), inter)
        y = x.clone()
        m.qk_norm_rope(y, None, pos.cuda(), freq.cuda(), interleaved=inter, q_out=y)
        assert torch.equal(o, y)
    o, _ = m.qk_norm_rope(x, None)
    assert torch.equal(o, x)
    z = torch.zeros(3, 2, D, dtype=torch.bfloat16, device="cuda")  # a row of zeros stays zero
    o, _ = m.qk_norm_rope(z, z, pos[:3].contiguous().cuda(), freq.cuda(), q_weight=w, k_weight=w)
    assert not o.float().abs().any()


def test_views_leave_the_rest_of_the_projection_alone():
    m = wlq()
    D, T = 128, 9
    qkv = _rows(8, T, 12, D).cuda()
    before = qkv.clone()
    pos, freq = _positions(1, T, 1, 500), _freq((64,))
    m.qk_norm_rope(qkv[:, :6], qkv[:, 6:9], pos.cuda(), freq.cuda(), q_out=qkv[:, :6], k_out=qkv[:, 6:9])
    assert torch.equal(qkv[:, 9:], before[:, 9:]) and not torch.equal(qkv[:, :9], before[:, :9])


def _batch(q_lens, kv_lens, page, seed, extra=2):
    per = max(1, max(-(-k // page) for k in kv_lens))
    pages = len(kv_lens) * per + extra
    perm = np.random.default_rng(seed).permutation(pages)[: len(kv_lens) * per].reshape(len(kv_lens), per).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    return cu, np.array(kv_lens, dtype=np.int32), perm, pages


def _dev(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


@pytest.mark.parametrize("D,group,page,heads", [(128, 128, 16, 8), (128, 32, 64, 1), (64, 64, 32, 3), (64, 32, 256, 5), (128, 64, 128, 32)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([1, 1, 1], [17, 300, 64]), ([70, 0, 5, 33], [70, 9, 200, 33])])
@pytest.mark.parametrize("rotate", [0, 1, 2])
def test_append_writes_the_exact_codes(D, group, page, heads, q_lens, kv_lens, rotate):
    m = wlq()
    cu, kv, table, pages = _batch(q_lens, kv_lens, page, 7)
    T = int(cu[-1])
    x = _rows(T + heads, T, 2 * heads, D).cuda()
    x[0, 0, :5] = 0.0
    x[-1, -1] = 0.0                                                      # an all-zero group
    x[0, -1] = torch.arange(D).bfloat16().cuda() % 14 - 7                  # whole steps of a unit scale, and
    x[0, -1, 1::2] += 0.5                                                # ties
    k, v = x[:, :heads], x[:, heads:]
    w = (1 + 0.2 * _rows(2, 1, 1, D, 0.0).reshape(D)).bfloat16().cuda() if rotate else None
    sections = (D // 4,) if rotate == 1 else (D // 8, D // 4, D // 8)
    pos, freq = _positions(3, T, len(sections), 100000), _freq(sections)
    rope = dict(positions=pos.cuda(), inv_freq=freq.cuda(), sections=sections, interleaved=rotate == 2) if rotate else {}
    cache = m.Kv4Cache(pages, heads, page, D, group)
    for t in cache:
        t.view(torch.uint8).fill_(0xA5)
    before = [t.clone() for t in cache]
    dcu, dkv, dtab = _dev(cu, kv, table)
    m.kv4_append(cache, k, v, dcu, dkv, dtab, max(q_lens), k_weight=w, **rope)
    m.check_status()
    kr = ref.f64(k)
    if rotate:
        kr = ref.key_bits(ref.norm_rope(kr, ref.f64(w), 1e-6, pos.numpy(), freq.numpy(), sections, rotate == 2))
    want = [t.cpu().numpy().copy() for t in before]
    for vals, ci, si in ((kr, 0, 1), (ref.f64(v), 2, 3)):
        q, s = ref.quantize4(vals, group)
        b4 = ref.pack4(q)
        for b in range(len(q_lens)):
            for i in range(q_lens[b]):
                p = kv_lens[b] - q_lens[b] + i
                want[ci][table[b][p // page], :, p % page] = b4[cu[b] + i]
                want[si][table[b][p // page], :, p % page] = s[cu[b] + i].astype(np.float16)
    for got, w_ in zip(cache, want):
        np.testing.assert_array_equal(got.cpu().numpy().view(np.uint8), w_.view(np.uint8))
    # and back as values
    kb, vb = m.kv4_read(cache, dcu, dkv, dtab, max(q_lens), T)
    for vals, o in ((kr, kb), (ref.f64(v), vb)):
        q, s = ref.quantize4(vals, group)
        np.testing.assert_array_equal(ref.f64(o), ref.bf16_rne((q.reshape(*s.shape, group) * s[..., None]).reshape(q.shape)))


def test_append_has_the_bits_of_quantize_ex_on_the_exact_keys():
    m = wlq()
    T, H, D, group, page = 50, 4, 128, 32, 64
    x = _rows(1, T, 2 * H, D).cuda()
    w = (1 + 0.2 * _rows(2, 1, 1, D, 0.0).reshape(D)).bfloat16().cuda()
    pos, freq = _positions(3, T, 1, 5000).cuda(), _freq((64,)).cuda()
    cu, kv, table = _dev(*_batch([T], [T], page, 1)[:3])
    cache = m.Kv4Cache(3, H, page, D, group)
    m.kv4_append(cache, x[:, :H], x[:, H:], cu, kv, table, T, pos, freq, k_weight=w)
    exact = ref.key_bits(ref.norm_rope(ref.f64(x[:, :H]), ref.f64(w), 1e-6, pos.cpu().numpy(), freq.cpu().numpy(), (64,), True))
    codes, scales = m.quantize_ex(torch.from_numpy(exact).bfloat16().cuda().reshape(T * H, D), 4, group, m.SCALE_F16)
    t = np.arange(T)
    pg = table.cpu().numpy()[0][t // page]
    got = cache[0].cpu().numpy()[pg, :, t % page]
    np.testing.assert_array_equal(ref.unpack4(got, D), codes.cpu().numpy().reshape(T, H, D))
    np.testing.assert_array_equal(cache[1].cpu().numpy()[pg, :, t % page], scales.cpu().numpy().reshape(T, H, -1))


def test_append_of_many_rows_has_the_exact_codes():
    """Enough keys (2 million) that values next to a border are among them: some 600 within fp32's error of one."""
    m = wlq()
    T, H, D, group, page = 1000, 16, 128, 128, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(T, 2 * H, D, generator=g, device="cuda") * (1 + 3 * (torch.rand(D, generator=g, device="cuda") > 0.95))).bfloat16()
    w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    pos, freq = _positions(3, T, 1, 1 << 20).cuda(), _freq((64,)).cuda()
    cu, kv, table = _dev(*_batch([T], [T], page, 1)[:3])
    cache = m.Kv4Cache(20, H, page, D, group)
    for inter in (True, False):
        m.kv4_append(cache, x[:, :H], x[:, H:], cu, kv, table, T, pos, freq, k_weight=w, interleaved=inter)
        exact = ref.key_bits(ref.norm_rope(ref.f64(x[:, :H]), ref.f64(w), 1e-6, pos.cpu().numpy(), freq.cpu().numpy(), (64,), inter))
        q, s = ref.quantize4(exact, group)
        t = np.arange(T)
        pg = table.cpu().numpy()[0][t // page]
        np.testing.assert_array_equal(ref.unpack4(cache[0].cpu().numpy()[pg, :, t % page], D), q)
        np.testing.assert_array_equal(cache[1].cpu().numpy()[pg, :, t % page].astype(np.float64), s)


def test_append_flags_values_that_do_not_fit():
    m = wlq()
    m.check_status()
    D, H, page = 64, 2, 16
    x = _rows(1, 3, 2 * H, D, 0.0).cuda()
    x[0, 0, 3] = float("nan")
    x[1, 3, 40] = float("inf")
    x[2, 2, 1] = 65536.0
    x[2, 3, 1] = 65280.0  # the largest that fits
    cu, kv, table = _dev(*_batch([3], [3], page, 1)[:3])
    cache = m.Kv4Cache(3, H, page, D, 32)
    m.kv4_append(cache, x[:, :H], x[:, H:], cu, kv, table, 3)
    assert m.get_status() == m.ERR_NONFINITE
    p = int(table[0, 0])
    for sc, tok, head, grp in ((1, 0, 0, 0), (3, 1, 1, 1), (3, 2, 0, 0)):
        assert float(cache[sc][p, head, tok, grp]) == 0.0
        codes = ref.unpack4(cache[sc - 1][p, head, tok].cpu().numpy(), D)
        assert not codes[32 * grp:32 * grp + 32].any()
    assert float(cache[3][p, 1, 2, 0]) * 7 < 65504 and float(cache[3][p, 0, 1, 0]) > 0
    m.check_status()


def test_offsets_out_of_range_are_skipped_and_reported():
    """Bad lengths and pages never reach memory: the kernel's own checks skip them (tests/test_kvslot.py runs the same rules on the host)."""
    m = wlq()
    D, H, page = 64, 1, 16
    x = _rows(1, 8, 2 * H, D, 0.0).cuda()
    for cu, kv, table, max_q in (
            ([0, 8], [4], [[0, 1]], 8),        # fewer cached tokens than tokens
            ([0, 8], [40], [[0, 1]], 8),       # past the table
            ([0, 8], [8], [[5, 1]], 8),        # a page outside the pool
            ([0, 8], [8], [[-1, 1]], 8),
            ([0, 9], [9], [[0, 1]], 9),        # more tokens than the tensors have
            ([4, 2], [8], [[0, 1]], 8),        # decreasing offsets
            ([0, 8], [8], [[0, 1]], 7)):       # more tokens than max_q
        cache = m.Kv4Cache(2, H, page, D, 32)
        a = [torch.tensor(t, dtype=torch.int32, device="cuda") for t in (cu, kv, table)]
        m.kv4_append(cache, x[:, :H], x[:, H:], *a, max_q)
        assert m.get_status() == m.ERR_INDEX, (cu, kv, table, max_q)
        m.check_status()


def test_two_streams_and_a_captured_append():
    m = wlq()
    T, H, D, group, page = 40, 4, 128, 64, 16
    x = _rows(1, T, 2 * H, D).cuda()
    pos, freq = _positions(3, T, 1, 5000).cuda(), _freq((64,)).cuda()
    cu, kv, table = _dev(*_batch([T], [T], page, 1)[:3])
    want = m.Kv4Cache(5, H, page, D, group)
    m.kv4_append(want, x[:, :H], x[:, H:], cu, kv, table, T, pos, freq)
    got = m.Kv4Cache(5, H, page, D, group)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.kv4_append(got, x[:, :H], x[:, H:], cu, kv, table, T, pos, freq)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for t in got:
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.kv4_append(got, x[:, :H], x[:, H:], cu, kv, table, T, pos, freq)
        back = m.kv4_read(got, cu, kv, table, T, T)
    for seed in (1, 2):
        x.copy_(_rows(seed, T, 2 * H, D))
        graph.replay()
        m.kv4_append(want, x[:, :H], x[:, H:], cu, kv, table, T, pos, freq)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all(torch.equal(a, b) for a, b in zip(back, m.kv4_read(want, cu, kv, table, T, T)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-60, 1e-40, 1e-30])
@pytest.mark.parametrize("inter", [False, True])
def test_rows_next_to_zero_are_normed(D, eps, inter):
    """Rows whose squares leave fp32 below, beside ordinary ones in the same warp, with an eps too small to hide them."""
    m = wlq()
    T, H = 12, 5
    x = _rows(D, T, H, D, 0.5).float()
    for t, size in enumerate((1e-12, 1e-18, 1e-20, 1e-22, 1e-25, 1e-30, 1e-36, 1e-38, 4e-39)):
        x[t, 1::2] *= size
    x = x.bfloat16()
    x[9, 2] = 0
    x[9, 2, 7] = 9.2e-41          # one smallest subnormal among zeros
    x[10, 3, 1:] *= 1e-25         # one ordinary value among tiny ones
    if eps:
        x[11, 0] = 0              # stays zero; with eps = 0 the formula is 0 / 0
    w = (1 + 0.3 * _rows(3, 1, 1, D, 0.0).reshape(D)).bfloat16()
    pos, freq = _positions(1, T, 1, 5000), _freq((D // 2,))
    args = ref.f64(x), ref.f64(w), eps
    o, k = m.qk_norm_rope(x.cuda(), x.cuda(), pos.cuda(), freq.cuda(), interleaved=inter, q_weight=w.cuda(), k_weight=w.cuda(), eps=eps)
    _check_rows(ref.f64(o), *args, pos.numpy(), freq.numpy(), (D // 2,), inter)
    assert torch.equal(o, k)
    o, _ = m.qk_norm_rope(x.cuda(), None, q_weight=w.cuda(), eps=eps)
    _check_rows(ref.f64(o), *args, None, None, None, True)
    # the same rows into the cache: exact codes, nothing flagged
    cu, kv, table = _dev(*_batch([T], [T], 16, 1)[:3])
    cache = m.Kv4Cache(3, H, 16, D, 32)
    m.kv4_append(cache, x.cuda(), x.cuda(), cu, kv, table, T, pos.cuda(), freq.cuda(), interleaved=inter, k_weight=w.cuda(), eps=eps)
    m.check_status()
    q, s = ref.quantize4(ref.key_bits(ref.norm_rope(*args, pos.numpy(), freq.numpy(), (D // 2,), inter)), 32)
    p = int(table[0, 0])
    np.testing.assert_array_equal(ref.unpack4(cache[0][p, :, :T].cpu().numpy().transpose(1, 0, 2), D), q)
    np.testing.assert_array_equal(cache[1][p, :, :T].cpu().numpy().transpose(1, 0, 2).astype(np.float64), s)


def _exact_turn(pos, f):
    """cos and sin of pos * f (both exact integers over powers of two), the angle reduced with 60 digits of pi."""
    from decimal import Decimal, localcontext
    with localcontext() as c:
        c.prec = 90

        def arctan_inverse(n):  # of 1 / n
            x, total, k = Decimal(1) / n, Decimal(0), 0
            while abs(x) > Decimal(10) ** -85:
                total += x / (2 * k + 1) if k % 2 == 0 else -x / (2 * k + 1)
                x /= n * n
                k += 1
            return total

        two_pi = 8 * (4 * arctan_inverse(5) - arctan_inverse(239))  # Machin
        a = Decimal(int(pos)) * Decimal(float(f))                   # exact: a float is a short decimal
        a -= two_pi * (a / two_pi).to_integral_value()
        return float(a)


def _far_keys(seed, D, inter, group):
    """Positions up to the ends of int32 and frequencies of full 24 bits: the angles have up to 55 bits.  Heads that hold one
    pair of inputs, such that the exact rotation and that of the angle rounded to 53 bits round to different keys."""
    g = np.random.default_rng(seed)
    pairs = D // 2
    freq = g.uniform(0.5, 1.0, pairs).astype(np.float32)
    pos = np.array([(1 << 31) - 1, -(1 << 31) + 1, (1 << 31) - 3, (1 << 30) + 7, 1234567891, -1987654321, 2147400001, 2000000011], dtype=np.int64)
    a, b = (t.ravel() for t in np.meshgrid(1 + np.arange(128) / 128, (1 + np.arange(128) / 128)[:, None] * np.array([-2, -1, 1, 2]), indexing="ij"))
    rows = []
    for t, p in enumerate(pos):
        for i in range(0, pairs, 2):
            w = [_exact_turn(p, freq[i]), _exact_turn(1, float(p) * float(freq[i]))]
            first, second = ([f(u) for u in w] for f in (lambda u: a * np.cos(u) - b * np.sin(u), lambda u: a * np.sin(u) + b * np.cos(u)))
            for y, other in ((first, second), (second, first)):
                hit = (ref.key_bits(y[0]) != ref.key_bits(y[1])) & (np.abs(y[0]) > np.abs(other[0]))  # the largest of its group: the scale changes
                rows += [(t, i, a[j], b[j], first[0][j], second[0][j]) for j in np.nonzero(hit)[0][:2]]
    T, H = len(pos), len(rows)
    x, y = np.zeros((T, H, D)), np.zeros((T, H, D))
    for h, (t, i, a_, b_, f_, s_) in enumerate(rows):
        at = [2 * i, 2 * i + 1] if inter else [i, i + pairs]
        x[t, h, at], y[t, h, at] = (a_, b_), (f_, s_)
    return pos.astype(np.int32), freq, x, *ref.quantize4(ref.key_bits(y), group)


@pytest.mark.parametrize("D,inter", [(128, True), (64, False)])
def test_append_at_the_ends_of_the_positions(D, inter):
    m = wlq()
    group = 32
    pos, freq, x, q, s = _far_keys(D, D, inter, group)
    T, H = x.shape[:2]
    assert H >= 12
    k = torch.from_numpy(x).bfloat16().cuda()
    cu, kv, table = _dev(*_batch([T], [T], 16, 1)[:3])
    cache = m.Kv4Cache(3, H, 16, D, group)
    m.kv4_append(cache, k, k, cu, kv, table, T, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), interleaved=inter)
    m.check_status()
    p = int(table[0, 0])
    np.testing.assert_array_equal(ref.unpack4(cache[0][p, :, :T].cpu().numpy().transpose(1, 0, 2), D), q)
    np.testing.assert_array_equal(cache[1][p, :, :T].cpu().numpy().transpose(1, 0, 2).astype(np.float64), s)
