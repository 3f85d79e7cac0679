"""Refusals of the attention layer's entry points that need no GPU: every
argument is checked before anything touches the device."""
import ctypes

import pytest

import weight_only_quantized_rtn_b200 as m

P = 1 << 20  # a 16-byte aligned address that is never dereferenced
I3 = ctypes.c_int32 * 3


def rope(**kw):
    a = dict(q=P, q_stride=1024, q_heads=8, k=P, k_stride=256, k_heads=2, tokens=4, head_dim=128, q_weight=None, k_weight=None, eps=1e-6,
             positions=P, axes=3, inv_freq=P, rotary_dim=128, sections=I3(22, 21, 21), interleaved=1, q_out=P, q_out_stride=1024, k_out=P,
             k_out_stride=256, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.lib.wlq_qk_norm_rope(*a.values())


@pytest.mark.parametrize("want,kw", [
    (m.ERR_UNSUPPORTED, dict(head_dim=96)), (m.ERR_SHAPE, dict(tokens=-1)), (m.ERR_SHAPE, dict(tokens=1 << 31)),
    (m.ERR_INVALID_ARG, dict(q=None)), (m.ERR_INVALID_ARG, dict(k_out=None)), (m.ERR_SHAPE, dict(q_heads=-1)),
    (m.ERR_ALIGN, dict(q=P + 8)), (m.ERR_ALIGN, dict(k_stride=260)), (m.ERR_SHAPE, dict(q_stride=1016)),
    (m.ERR_SHAPE, dict(axes=0)), (m.ERR_SHAPE, dict(axes=5)), (m.ERR_SHAPE, dict(rotary_dim=120)), (m.ERR_SHAPE, dict(rotary_dim=144)),
    (m.ERR_SHAPE, dict(rotary_dim=0)), (m.ERR_INVALID_ARG, dict(inv_freq=None)), (m.ERR_INVALID_ARG, dict(sections=None)),
    (m.ERR_SHAPE, dict(sections=I3(22, 21, 22))), (m.ERR_SHAPE, dict(sections=I3(-1, 44, 21))), (m.ERR_ALIGN, dict(positions=P + 2)),
    (m.ERR_ALIGN, dict(q_weight=P + 1)), (m.ERR_INVALID_ARG, dict(eps=-1.0)), (m.ERR_INVALID_ARG, dict(eps=float("nan"))),
    (m.ERR_INVALID_ARG, dict(q_out_stride=2048)),
])
def test_norm_rope_refuses(want, kw):
    assert rope(**kw) == want
    assert m.lib.wlq_last_error()


def test_norm_rope_of_nothing_is_a_no_op():
    assert rope(tokens=0) == m.OK
    assert rope(q_heads=0, k_heads=0, q=None, k=None, q_out=None, k_out=None) == m.OK


def append(**kw):
    a = dict(k=P, k_stride=512, v=P, v_stride=512, tokens=4, heads=4, head_dim=128, k_weight=None, eps=1e-6, positions=None, axes=0, inv_freq=None,
             rotary_dim=0, sections=None, interleaved=1, cu=P, kv=P, batch=2, max_q=2, table=P, width=3, kc=P, ks=P, vc=P, vs=P, pages=8,
             page_size=16, group=64, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.lib.wlq_kv4_append(*a.values())


BAD_CACHE = [
    (m.ERR_UNSUPPORTED, dict(head_dim=256)), (m.ERR_UNSUPPORTED, dict(group=16)), (m.ERR_UNSUPPORTED, dict(head_dim=64, group=128)),
    (m.ERR_UNSUPPORTED, dict(page_size=8)), (m.ERR_UNSUPPORTED, dict(page_size=48)), (m.ERR_UNSUPPORTED, dict(page_size=512)),
    (m.ERR_INVALID_ARG, dict(kc=None)), (m.ERR_ALIGN, dict(vs=P + 4)), (m.ERR_INVALID_ARG, dict(cu=None)), (m.ERR_INVALID_ARG, dict(table=None)),
    (m.ERR_INVALID_ARG, dict(batch=-1)), (m.ERR_INVALID_ARG, dict(max_q=-1)), (m.ERR_SHAPE, dict(batch=1 << 16, max_q=1 << 16)),
    (m.ERR_ALIGN, dict(kv=P + 1)), (m.ERR_SHAPE, dict(heads=0)), (m.ERR_SHAPE, dict(pages=-1)),
]


@pytest.mark.parametrize("want,kw", BAD_CACHE + [(m.ERR_INVALID_ARG, dict(v=None)), (m.ERR_ALIGN, dict(v=P + 2)), (m.ERR_SHAPE, dict(k_stride=504))])
def test_append_refuses(want, kw):
    assert append(**kw) == want


def test_append_of_nothing_is_a_no_op():
    assert append(batch=0) == m.OK and append(max_q=0) == m.OK and append(tokens=0) == m.OK


def read(**kw):
    a = dict(cu=P, kv=P, batch=2, max_q=2, table=P, width=3, kc=P, ks=P, vc=P, vs=P, pages=8, page_size=16, group=64, tokens=4, heads=4,
             head_dim=128, k_out=P, v_out=P, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.lib.wlq_kv4_read(*a.values())


@pytest.mark.parametrize("want,kw", BAD_CACHE + [(m.ERR_INVALID_ARG, dict(v_out=None)), (m.ERR_ALIGN, dict(k_out=P + 8))])
def test_read_refuses(want, kw):
    assert read(**kw) == want


def attend(**kw):
    a = dict(q=P, q_stride=1024, tokens=4, q_heads=8, kv_heads=4, head_dim=128, cu=P, kv=P, batch=2, max_q=2, max_kv=100, table=P, width=3,
             kc=P, ks=P, vc=P, vs=P, pages=8, page_size=16, group=64, scale=0.1, causal=1, window=0, out=P, lse=None, ws=P, ws_bytes=1 << 40,
             stream=None)
    heads = kw.pop("heads", None)
    if heads is not None:
        kw["kv_heads"] = heads
    assert set(kw) <= set(a)
    a.update(kw)
    return m.lib.wlq_kv4_attention(*a.values())


@pytest.mark.parametrize("want,kw", BAD_CACHE + [
    (m.ERR_SHAPE, dict(q_heads=6)), (m.ERR_SHAPE, dict(q_heads=0)), (m.ERR_SHAPE, dict(q_heads=2)), (m.ERR_INVALID_ARG, dict(q=None)),
    (m.ERR_ALIGN, dict(q=P + 2)), (m.ERR_INVALID_ARG, dict(out=None)), (m.ERR_ALIGN, dict(out=P + 8)), (m.ERR_ALIGN, dict(lse=P + 2)),
    (m.ERR_INVALID_ARG, dict(scale=float("nan"))), (m.ERR_INVALID_ARG, dict(scale=float("inf"))), (m.ERR_INVALID_ARG, dict(window=-1)),
    (m.ERR_INVALID_ARG, dict(window=8, causal=0)), (m.ERR_INVALID_ARG, dict(max_kv=-1)),
    (m.ERR_WORKSPACE, dict(max_kv=100000, ws=None)), (m.ERR_WORKSPACE, dict(max_kv=100000, ws_bytes=16)), (m.ERR_ALIGN, dict(max_kv=100000, ws=P + 8)),
])
def test_attention_refuses(want, kw):
    assert attend(**kw) == want


def test_attention_of_nothing_is_a_no_op():
    assert attend(batch=0) == m.OK and attend(max_q=0) == m.OK and attend(tokens=0) == m.OK


def test_attention_workspace():
    f = m.kv4_attention_workspace
    assert f(0, 1, 1, 100, 8, 8, 128) == 0 and f(1, 1, 1, 100, 8, 3, 128) == 0 and f(1, 1, 1, 100, 8, 8, 96) == 0
    assert f(1, 1, 1, 64, 8, 8, 128) == 0                      # too short to split
    assert f(1, 1, 1, 1 << 20, 8, 8, 128) >= 8 * 2 * (128 + 2) * 4  # at least two parts a row


def int8(**kw):
    a = dict(xq=P, xs=P, M=4, wq=P, ws=P, N=64, K=128, bias=None, y=P, y_dtype=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.lib.wlq_int8_linear(*a.values())


def w8a8(**kw):
    a = dict(xq=P, M=4, wq=P, ws=P, N=64, K=128, bias=None, y=P, y_dtype=0, workspace=P, ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.lib.wlq_w8a8_linear(*a.values())


BAD_INT8 = [
    (m.ERR_INVALID_ARG, dict(M=-1)), (m.ERR_INVALID_ARG, dict(N=-1)), (m.ERR_SHAPE, dict(K=0)), (m.ERR_SHAPE, dict(K=24)),
    (m.ERR_SHAPE, dict(K=131072)), (m.ERR_INVALID_ARG, dict(y_dtype=2)), (m.ERR_INVALID_ARG, dict(xq=None)), (m.ERR_INVALID_ARG, dict(wq=None)),
    (m.ERR_INVALID_ARG, dict(ws=None)), (m.ERR_INVALID_ARG, dict(y=None)), (m.ERR_ALIGN, dict(xq=P + 8)), (m.ERR_ALIGN, dict(wq=P + 4)),
    (m.ERR_ALIGN, dict(ws=P + 2)), (m.ERR_ALIGN, dict(y=P + 2)), (m.ERR_ALIGN, dict(bias=P + 1)), (m.ERR_SHAPE, dict(M=1 << 31)),
    (m.ERR_SHAPE, dict(M=1 << 30, N=1 << 30)),
]


@pytest.mark.parametrize("want,kw", BAD_INT8 + [(m.ERR_INVALID_ARG, dict(xs=None)), (m.ERR_ALIGN, dict(xs=P + 2))])
def test_int8_refuses(want, kw):
    assert int8(**kw) == want


@pytest.mark.parametrize("want,kw", BAD_INT8 + [(m.ERR_WORKSPACE, dict(workspace=None)), (m.ERR_WORKSPACE, dict(ws_bytes=100)),
                                                (m.ERR_ALIGN, dict(workspace=P + 8))])
def test_w8a8_refuses(want, kw):
    assert w8a8(**kw) == want


def test_int8_of_nothing_is_a_no_op():
    assert int8(M=0) == m.OK and int8(N=0) == m.OK and w8a8(M=0) == m.OK and w8a8(N=0) == m.OK
    assert m.w8a8_workspace(4, 128) >= 4 * 128 + 16 and m.w8a8_workspace(0, 128) == 0 and m.w8a8_workspace(4, 24) == 0


def test_caches_copy_and_save():
    import copy
    import pickle

    cache = m.Kv4Cache(3, 2, 16, 64, 32, device="cpu")
    for again in (copy.copy(cache), copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        assert [(t.shape, t.dtype) for t in again] == [(t.shape, t.dtype) for t in cache]


def test_every_status_has_its_name():
    import os
    import re

    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(m.__file__))), "include", "wlq.h")).read()
    names = {int(v): n for n, v in re.findall(r"(WLQ_(?:OK|ERR_\w+)) = (\d+)", header)}
    assert names == m.STATUS_NAMES
    assert "WLQ_ERR_INDEX" in str(m.WlqError(m.ERR_INDEX, "x"))


@pytest.mark.parametrize("scale", [2.1e38, -3.4e38])
def test_scales_whose_power_of_two_form_leaves_fp32_are_refused(scale):
    assert attend(scale=scale) == m.ERR_INVALID_ARG


def test_a_bound_beyond_every_length_plans_like_the_largest_length():
    f = m.kv4_attention_workspace
    for rows in (1, 64):
        assert f(rows, 1, rows, (1 << 63) - 1, 8, 8, 128) == f(rows, 1, rows, 1 << 31, 8, 8, 128) > 0


@pytest.mark.parametrize("name,kw", [("max_q", dict(max_q=(1 << 32) + 1)), ("max_q", dict(max_q=-1)), ("window", dict(window=(1 << 32) + 3)),
                                     ("window", dict(window=-(1 << 32)))])
def test_bounds_that_32_bits_do_not_hold_are_refused(name, kw, monkeypatch):
    """They would reach the library as their lower 32 bits."""
    import torch

    monkeypatch.setattr(m, "_on", lambda *a: None)
    cache = m.Kv4Cache(3, 2, 16, 64, 32, device="cpu")
    i32 = [torch.zeros(n, dtype=torch.int32) for n in (2, 1)] + [torch.zeros(1, 3, dtype=torch.int32)]
    a = dict(max_q=1, max_kv=4)
    a.update(kw)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(m.WlqError, match=name):
        m.kv4_attention(q, cache, *i32, **a)
    if name == "max_q":
        with pytest.raises(m.WlqError, match=name):
            m.kv4_append(cache, q, q, *i32, a["max_q"])
        with pytest.raises(m.WlqError, match=name):
            m.kv4_read(cache, *i32, a["max_q"], 1)
