"""kv4_attention against the 64-bit form (tests/attention_ref.py).

Bounds, from the roundings the header names.  Keys, values and weights enter
the products as fp16 (2^-11 relative each), scores and sums are fp32, the
output is rounded to bf16 (2^-8).  With E the largest possible score error of a
query, max_j scale sum_d |q_d k_jd| (2^-11 + 2^-20), A = sum_j p_j |v_j| and
B = 2^-25 sum_j |q_j| max_j s_j (q, s: the values' codes and scales):
    |out - ref| <= 2^-8 |ref| + (A (2 E + 2 * 2^-11 + 2^-16) + B) (1 + 2^-8),
    |lse - ref| <= E + 2^-16 max(1, |ref|)
(a weight's relative error is at most e^(2 E) - 1 after normalising; a weight
below 2^-14 of the running maximum's is an fp16 subnormal, whose half step is
2^-25, and the sum the weights are divided by is at least 1; where a weight
carries its value's scale it is held against the largest scale: B; 2^-16
covers ex2.approx and the fp32 sums of at most 2^16 terms' worth of rounding).
For random values the errors average out: the 2-norm error stays below 2^-8
of the result's (2^-8 / sqrt 3 from the output's rounding, 2^-11 each from the
other roundings, added in squares)."""
import numpy as np
import pytest
import torch

from tests import attention_ref as ref

pytestmark = pytest.mark.gpu


def wlq():
    import weight_only_quantized_rtn_b200 as m
    return m


def make(seed, q_lens, kv_lens, hk, share, D, group, page, extra_pages=3, pool=None, tail=0):
    """Random cache on scattered pages; places no sequence owns hold NaN scales, rows of no sequence NaN queries."""
    g = torch.Generator().manual_seed(seed)
    per = max(1, max(-(-k // page) for k in kv_lens))
    pages = pool or len(kv_lens) * per + extra_pages
    table = torch.randperm(pages, generator=g)[: len(kv_lens) * per].reshape(len(kv_lens), per).to(torch.int32)
    if pool:  # the last pages of a large pool
        table = (pool - 1 - torch.randperm(len(kv_lens) * per, generator=g)).reshape(len(kv_lens), per).to(torch.int32)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T = int(cu[-1]) + tail
    m = wlq()
    cache = m.Kv4Cache(pages, hk, page, D, group)
    if not pool:
        for t in (cache[1], cache[3]):
            t.fill_(float("nan"))
        for t in (cache[0], cache[2]):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for b, kv in enumerate(kv_lens):
        j = torch.arange(kv)
        pg, place = table[b, j // page].long().cuda(), (j % page).cuda()
        for ci, spread in ((0, 2.0), (2, 1.0)):
            x = torch.randn(kv, hk, D, generator=g) * torch.exp(0.5 * spread * torch.randn(kv, hk, 1, generator=g))
            c, s = ref.quantize4(ref.f64(x.bfloat16()), group)
            cache[ci][pg, :, place] = torch.from_numpy(ref.pack4(c)).cuda()
            cache[ci + 1][pg, :, place] = torch.from_numpy(s.astype(np.float16)).cuda()
    q = torch.randn(T, hk * share, D, generator=g).bfloat16()
    q[int(cu[-1]):] = float("nan")
    return q.cuda(), cache, cu, np.array(kv_lens, dtype=np.int32), table.numpy()


def check(m, q, cache, cu, kv, table, hk, causal, window, scale=None, max_q=None, max_kv=None, ws=None, random=True):
    T, Hq, D = q.shape
    dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (cu, kv, table)]
    out = torch.full((T, Hq, D), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), -7.0, device="cuda")
    max_q = int(max(np.diff(cu))) if max_q is None else max_q
    max_kv = int(max(kv)) if max_kv is None else max_kv
    m.kv4_attention(q, cache, *dev, max_q, max_kv, scale=scale, causal=causal, window=window, out=out, lse=lse, workspace=ws)
    sc = D ** -0.5 if scale is None else scale
    n = int(cu[-1])
    r = ref.attention(q, cache, cu, kv, table, sc, causal, window)
    want, want_lse, E, A, B = (r[k][:n] for k in ("out", "lse", "E", "A", "B"))
    got, got_lse = ref.f64(out), ref.f64(lse)
    assert (got[n:] == -7).all() and (got_lse[n:] == -7).all()  # rows of no sequence
    got, got_lse = got[:n], got_lse[:n]
    tol = 2.0 ** -8 * np.abs(want) + (A * (np.expm1(2 * E) + 2.0 ** -10 + 2.0 ** -16)[..., None] + B) * (1 + 2.0 ** -8)
    err = np.abs(got - want)
    assert (err <= tol).all(), "%r" % ((np.nanmax(err / tol), np.unravel_index(np.nanargmax(err / tol), err.shape)),)
    none = np.isneginf(want_lse)
    assert (np.isneginf(got_lse) == none).all() and (got[none] == 0).all()
    el = np.abs(got_lse[~none] - want_lse[~none])
    assert (el <= E[~none] + 2.0 ** -16 * np.maximum(1, np.abs(want_lse[~none]))).all()
    if random and n * Hq >= 8:
        assert np.linalg.norm(got - want) <= 2.0 ** -8 * np.linalg.norm(want)
    return out, lse


@pytest.mark.parametrize("D,group,page", [(128, 32, 16), (128, 64, 64), (128, 128, 256), (64, 32, 32), (64, 64, 128)])
@pytest.mark.parametrize("hk,share", [(1, 1), (2, 4), (3, 8), (1, 12), (2, 16)])
def test_single_tokens(D, group, page, hk, share):
    m = wlq()
    kv = [1, 15, 16, 17, 33, 300]
    a = make(hk * share + D, [1] * len(kv), kv, hk, share, D, group, page, tail=2)
    check(m, *a, hk, True, 0)
    m.check_status()


@pytest.mark.parametrize("D,page", [(128, 16), (64, 64)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 7), (True, 130), (True, 100000)])
@pytest.mark.parametrize("share", [1, 4])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([5, 0, 1, 20], [5, 0, 90, 44]), ([37, 129], [200, 129]), ([3, 1, 2], [3, 700, 260])])
def test_chunks(D, page, causal, window, share, q_lens, kv_lens):
    m = wlq()
    a = make(sum(q_lens) + share, q_lens, kv_lens, 2, share, D, 32, page, tail=1)
    check(m, *a, 2, causal, window)
    m.check_status()


@pytest.mark.parametrize("D,group,page", [(128, 32, 16), (128, 128, 64), (64, 64, 256), (64, 32, 32)])
@pytest.mark.parametrize("share,q_lens,kv_lens", [
    (1, [129], [129]), (1, [600, 40], [600, 1500]), (4, [64, 1, 300], [128, 5, 900]), (8, [33, 257], [2000, 257]), (3, [100], [3000])])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 200)])
def test_prompts_and_chunks_of_many_rows(D, group, page, share, q_lens, kv_lens, causal, window):
    m = wlq()
    a = make(sum(kv_lens) + share, q_lens, kv_lens, 2, share, D, group, page, tail=3)
    out, _ = check(m, *a, 2, causal, window)
    again, _ = check(m, *a, 2, causal, window)
    assert torch.equal(out, again)
    m.check_status()


@pytest.mark.parametrize("kv,window", [(5000, 0), (20011, 0), (20011, 600)])
def test_long_caches_are_split(kv, window):
    m = wlq()
    a = make(kv, [1, 1], [kv, 40], 1, 4, 128, 64, 128)
    assert m.kv4_attention_workspace(2, 2, 1, kv, 4, 1, 128) > 0
    out, lse = check(m, *a, 1, True, window)
    again, _ = check(m, *a, 1, True, window, ws=torch.full((m.kv4_attention_workspace(2, 2, 1, kv, 4, 1, 128),), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out, again)  # reproducible, whatever the workspace held
    check(m, *a, 1, True, window, max_kv=1)      # wrong bounds of the lengths cost speed, not results
    check(m, *a, 1, True, window, max_kv=1 << 20)
    check(m, *a, 1, True, window, max_q=3)
    m.check_status()


@pytest.mark.parametrize("D,group,page", [(128, 64, 64), (64, 32, 16)])
@pytest.mark.parametrize("share,max_q", [(4, 1), (3, 4), (8, 4)])
@pytest.mark.parametrize("longest", [600, 799, 1100, 1400, 1800, 2100])
def test_parts_joined_without_a_workspace(D, group, page, share, max_q, longest):
    """Two to eight short parts a sequence: some hold nothing (short and empty sequences, a window, bad pages)."""
    m = wlq()
    a = make(longest, [1, max_q, max_q - 1, 1, max_q], [longest, longest - 37, max_q - 1, 33, longest // 2], 2, share, D, group, page)
    assert m.kv4_attention_workspace(a[0].shape[0], 5, max_q, longest, 2 * share, 2, D) == 0
    for causal, window in ((True, 0), (False, 0), (True, 50)):
        check(m, *a, 2, causal, window)
    m.check_status()
    a[4][1, 2:-1] = -1
    check(m, *a, 2, True, 0, random=False)
    assert m.get_status() == m.ERR_INDEX
    m.check_status()


@pytest.mark.parametrize("D,group,page", [(128, 64, 64), (64, 32, 16)])
@pytest.mark.parametrize("hk,share,q_lens,kv_lens", [
    (50, 1, [520, 40], [1100, 700]), (13, 4, [200, 0, 130], [1300, 0, 260]), (80, 1, [40, 33], [6400, 6161]), (80, 1, [40], [6400])])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 300)])
def test_the_last_round_of_row_tiles_is_split(D, group, page, hk, share, q_lens, kv_lens, causal, window):
    """More row tiles than SMs, a part of them in pieces: short and empty sequences among them, rows behind the last."""
    m = wlq()
    a = make(hk + D, q_lens, kv_lens, hk, share, D, group, page, tail=3)
    check(m, *a, hk, causal, window)
    m.check_status()


def test_scores_that_grow_move_the_maximum():
    """Keys whose scores climb by far more than the lazy maximum's 2^8, then fall; the largest last, first and in between."""
    m = wlq()
    D, n = 64, 257
    for order, n_q in ((np.arange(n), 3), (np.arange(n)[::-1].copy(), 3), (np.abs(np.arange(n) - 128), 3), (np.arange(n), 90),
                       (np.arange(n)[::-1].copy(), 90), (np.abs(np.arange(n) - 128), 90)):
        q, cache, cu, kv, table = make(11, [n_q], [n], 1, 2, D, 32, 16)
        pages = table[0]
        for j in range(n):
            s = np.float16(0.02 * (order[j] + 1))
            cache[1][pages[j // 16], 0, j % 16] = torch.tensor(s)
            cache[0][pages[j // 16], 0, j % 16] = torch.from_numpy(ref.pack4(np.full(D, 7, dtype=np.int8))).cuda()
        q.abs_()
        check(m, q, cache, cu, kv, table, 1, False, 0, scale=1.0, random=False)
        check(m, q, cache, cu, kv, table, 1, False, 0, scale=-1.0, random=False)


def test_scale_zero_and_wide_queries():
    m = wlq()
    a = make(3, [2, 9], [50, 9], 2, 4, 128, 64, 16)
    check(m, *a, 2, True, 0, scale=0.0)
    q = a[0].clone()
    q[0, 0] *= 1e30     # large and tiny rows: their power of two is taken out and put back
    q[1, 1] *= 1e-30
    check(m, q, *a[1:], 2, True, 0, scale=1e-30, random=False)
    q = a[0].clone()
    q[:] = 0
    check(m, q, *a[1:], 2, True, 0)


def test_query_views_and_reproducible():
    m = wlq()
    q, cache, cu, kv, table = make(5, [4, 7], [60, 7], 2, 4, 128, 64, 16)
    wide = torch.zeros(11, 3 * 8 * 128, dtype=torch.bfloat16, device="cuda")
    wide[:, : 8 * 128] = q.reshape(11, -1)
    dev = [torch.from_numpy(x).cuda() for x in (cu, kv, table)]
    a = m.kv4_attention(q, cache, *dev, 7, 60)
    b = m.kv4_attention(wide[:, : 8 * 128].view(11, 8, 128), cache, *dev, 7, 60)
    assert torch.equal(a, b)


def test_a_cache_beyond_four_gigabytes():
    """Pages whose codes lie past 2^32 bytes."""
    m = wlq()
    pool = 70000
    a = make(9, [1, 2], [130, 200], 8, 4, 128, 128, 128, pool=pool)
    assert a[1][0].numel() > 1 << 32
    check(m, *a, 8, True, 0)
    m.check_status()


def test_pages_out_of_range_count_as_not_seen():
    m = wlq()
    for q_lens in ([1, 1], [30, 40]):
        q, cache, cu, kv, table = make(6, q_lens, [64, 40], 1, 2, 64, 32, 16)
        table = table.copy()
        table[0, 1] = -1
        table[0, 2] = cache[0].shape[0]
        table[1, :] = 1 << 30
        check(m, q, cache, cu, kv, table, 1, True, 0, random=False)
        assert m.get_status() == m.ERR_INDEX
    # a table narrower than the sequence
    check_table = torch.from_numpy(table[:, :1].copy()).cuda()
    m.kv4_attention(q, cache, torch.from_numpy(cu).cuda(), torch.from_numpy(kv).cuda(), check_table, 1, 64)
    assert m.get_status() == m.ERR_INDEX
    m.check_status()


def test_lengths_out_of_range_are_skipped():
    m = wlq()
    q, cache, cu, kv, table = make(6, [3, 2], [64, 40], 1, 2, 64, 32, 16)
    for c, k, max_q in (([0, 3, 6], [64, 40], 3), ([0, 3, 5], [2, 40], 3), ([0, 3, 5], [64, 40], 2), ([-1, 3, 5], [64, 40], 4)):
        out = torch.full_like(q, -7.0)
        m.kv4_attention(q, cache, torch.tensor(c, dtype=torch.int32, device="cuda"), torch.tensor(k, dtype=torch.int32, device="cuda"),
                        torch.from_numpy(table).cuda(), max_q, 64, out=out)
        assert m.get_status() == m.ERR_INDEX
        bad = [r for b in range(2) for r in range(max(c[b], 0), min(c[b + 1], 5))
               if c[b] < 0 or c[b + 1] > 5 or k[b] < c[b + 1] - c[b] or c[b + 1] - c[b] > max_q]
        assert bad and (out[bad] == -7).all()
        good = [r for r in range(5) if r not in bad]
        assert (out[good] != -7).any()


def test_streams_and_graphs():
    m = wlq()
    q, cache, cu, kv, table = make(8, [1, 1], [3000, 500], 2, 4, 128, 64, 64)
    dev = [torch.from_numpy(x).cuda() for x in (cu, kv, table)]
    want = m.kv4_attention(q, cache, *dev, 1, 3000)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for s in (s1, s2):  # two calls at once, a workspace each
        with torch.cuda.stream(s):
            outs.append(m.kv4_attention(q, cache, *dev, 1, 3000))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = m.kv4_attention(q, cache, *dev, 1, 3000)
    with torch.cuda.graph(g2):
        o2 = m.kv4_attention(q, cache, *dev, 1, 3000)
    q.copy_(q.flip(0))
    want = m.kv4_attention(q, cache, *dev, 1, 3000)
    for _ in range(2):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, want) and torch.equal(o2, want)
    dev[1].fill_(64)  # the lengths are read when the graph runs
    g1.replay()
    assert torch.equal(o1, m.kv4_attention(q, cache, *dev, 1, 3000))


def test_lengths_past_the_table_end_at_once():
    """A length the table has no room for (up to 2^31 - 1): its tokens count as not seen, and nobody walks them."""
    m = wlq()
    for n in (1, 50):
        q, cache, cu, kv, table = make(6, [n, 1], [64, 40], 1, 2, 64, 32, 16)
        dev = [torch.from_numpy(x).cuda() for x in (cu, kv, table)]
        want = m.kv4_attention(q, cache, *dev, n, 64, causal=False)
        dev[1][0] = (1 << 31) - 1
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        got = m.kv4_attention(q, cache, *dev, n, 64, causal=False)
        end.record()
        assert m.get_status() == m.ERR_INDEX
        assert torch.equal(got, want)  # not causal: all of the table's tokens
        assert start.elapsed_time(end) < 100
        dev[1][0] = 0
    m.check_status()


def test_calls_on_a_given_stream():
    m = wlq()
    q, cache, cu, kv, table = make(8, [1, 1], [3000, 500], 2, 4, 128, 64, 64)
    dev = [torch.from_numpy(x).cuda() for x in (cu, kv, table)]
    want = m.kv4_attention(q, cache, *dev, 1, 3000)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [m.kv4_attention(q, cache, *dev, 1, 3000, stream=s) for _ in range(20)]
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(20)]  # may not take the calls' workspaces
    s.synchronize()
    assert all(torch.equal(o, want) for o in got) and len(junk) == 20


def test_tensors_elsewhere_and_of_other_shapes_are_refused():
    m = wlq()
    q, cache, cu, kv, table = make(8, [1], [30], 2, 4, 64, 32, 16)
    dev = [torch.from_numpy(x).cuda() for x in (cu, kv, table)]
    bad = [
        (q.cpu(), cache, *dev), (q.float(), cache, *dev), (q[0], cache, *dev), (q[:, :, :32], cache, *dev), (q[:, :3], cache, *dev),
        (q, (cache[0].cpu(),) + tuple(cache[1:]), *dev), (q, (cache[0], cache[1].float()) + tuple(cache[2:]), *dev),
        (q, (cache[0][..., :16], *cache[1:]), *dev), (q, cache, dev[0].long(), dev[1], dev[2]), (q, cache, dev[0][:1], dev[1], dev[2]),
        (q, cache, dev[0], dev[1], dev[2][0]), (q.transpose(1, 2).contiguous().transpose(1, 2), cache, *dev),
    ]
    for args in bad:
        with pytest.raises(m.WlqError):
            m.kv4_attention(*args, 1, 30)
    with pytest.raises(m.WlqError):
        m.kv4_attention(q, cache, *dev, 1, 30, out=torch.empty_like(q).float())
    with pytest.raises(m.WlqError):
        m.kv4_attention(q, cache, *dev, 1, 30, lse=torch.empty(1, 8, device="cuda").half())
    with pytest.raises(m.WlqError):
        m.qk_norm_rope(q, None, torch.zeros(2, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda"))
    with pytest.raises(m.WlqError):
        m.qk_norm_rope(q, None, torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(m.WlqError):
        m.qk_norm_rope(None, None)
    with pytest.raises(m.WlqError):
        m.w8a8_linear(torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 32, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda"))
    with pytest.raises(m.WlqError):
        m.w8a8_linear(torch.zeros(2, 24, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 24, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda"))


def test_workspaces_that_are_views_of_less_memory_are_refused():
    m = wlq()
    q, cache, cu, kv, table = make(8, [1, 1], [30, 20], 2, 4, 64, 32, 16)
    dev = [torch.from_numpy(x).cuda() for x in (cu, kv, table)]
    n = m.kv4_attention_workspace(2, 2, 1, 1 << 20, 8, 2, 64)
    assert n > 0
    ws = torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)
    with pytest.raises(m.WlqError, match="contiguous"):
        m.kv4_attention(q, cache, *dev, 1, 1 << 20, workspace=ws)
    x, wq, s = torch.zeros(4, 128, device="cuda").bfloat16(), torch.zeros(16, 128, dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda")
    with pytest.raises(m.WlqError, match="contiguous"):
        m.w8a8_linear(x, wq, s, workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(m.w8a8_workspace(4, 128)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("size", [1e-33, 1e-36, 2e-39, 9.2e-41])
def test_queries_next_to_zero(D, n, size):
    """Rows whose largest value is next to bf16's smallest, with zeros in them (9.2e-41 is the smallest subnormal): nearly
    the mean of the values, at a scale that hardly matters and at one that lifts the scores."""
    m = wlq()
    q, *a = make(D + n, [n, 1], [n + 300, 70], 2, 2, D, 32, 16)
    q = q.clone()
    small = (torch.rand(q.shape, generator=torch.Generator().manual_seed(1)) * size).cuda().bfloat16()
    q[0] = small[0]
    q[-1, 1:] = small[-1, 1:]
    q[0, :, ::3] = 0
    q[-1, 1, 1:] = 0
    q[-1, 1, 0] = size
    assert torch.isfinite(q).all() and float(q[0].float().abs().max()) > 0
    check(m, q, *a, 2, True, 0, random=False)
    m.check_status()
    q[:] = small
    check(m, q, *a, 2, True, 0, scale=0.01 / size if size > 1e-38 else 1e38, random=False)
    m.check_status()


@pytest.mark.parametrize("D,group,page", [(128, 32, 16), (128, 128, 64), (64, 64, 32), (64, 32, 128)])
@pytest.mark.parametrize("n,share", [(1, 4), (3, 8), (50, 1), (70, 4)])
@pytest.mark.parametrize("back", ["none", "past", "other"])
def test_pages_given_back_behind_the_window(D, group, page, n, share, back):
    """Table entries of pages that no query sees: none (-1), past the pool, or a page that now holds something else, whose
    scales are not finite.  They are not read: the result is that of the whole cache, without an error."""
    m = wlq()
    m.check_status()
    for kv in (n + 90, n + 700, n + 701, n + 1663):
        for window in (1, 33, 80, 600):
            q, cache, cu, kvs, table = make(kv + share, [n, 1], [kv, 5], 2, share, D, group, page, tail=1)
            first = max(0, kv - n - window + 1)  # the first token that is seen
            table = table.copy()
            table[0, : first // page] = -1 if back == "none" else cache[0].shape[0]
            if back == "other":
                spare = next(p for p in range(cache[0].shape[0]) if p not in table)
                table[0, : first // page] = spare
                cache[1][spare] = float("nan")
                cache[3][spare] = float("nan")
                zero = [t.clone() for t in cache]  # the reference multiplies by zero weights: finite values there
                zero[1][spare] = 0
                zero[3][spare] = 0
                dev = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (cu, kvs, table)]
                got = m.kv4_attention(q, cache, *dev, n, kv, window=window)
                want, _ = check(m, q, zero, cu, kvs, table, 2, True, window, random=False)
                assert torch.equal(got[: n + 1], want[: n + 1])
            else:
                check(m, q, cache, cu, kvs, table, 2, True, window, random=False)
            m.check_status()
    if back != "other":  # a page that is seen is still reported
        table[0, first // page] = -1
        check(m, q, cache, cu, kvs, table, 2, True, window, random=False)
        assert m.get_status() == m.ERR_INDEX


@pytest.mark.parametrize("n", [1, 40])
def test_a_sequence_of_as_many_tokens_as_a_length_holds(n):
    """2^31 - 1 cached tokens (one page over and over, another at the end): the place after the last token is not one."""
    m = wlq()
    D, page, kv = 64, 256, (1 << 31) - 1
    cache = m.Kv4Cache(2, 1, page, D, 64)
    cache[0].fill_(0x11)                     # the same low score for every token (a place without one would have 0)
    cache[1].fill_(1.0)
    cache[2].fill_(0x99)                     # values of one
    cache[3].fill_(1.0)
    cache[1][1, :, -1] = float("nan")        # what no token was written to
    cache[3][1, :, -1] = float("nan")
    cache[2][1, :, -1] = 0
    table = torch.zeros(1, 1 << 23, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.ones(n, 1, D, dtype=torch.bfloat16, device="cuda")
    cu, kvs = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [kv]))
    o = m.kv4_attention(q, cache, cu, kvs, table, n, kv, causal=False)
    m.check_status()
    assert (o == 1).all()                    # sums of ones: exact, each accumulator has less than 2^24 of them (or steps of 16)
