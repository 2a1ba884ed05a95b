"""Paged cache and cross attention without a GPU: every refusal comes before the
first CUDA call, the rotary frequencies are plain host arithmetic, and the
binding's structs mirror the header's."""

import ctypes as C

import numpy as np
import pytest

import autoregressive_speech_token_gb300 as pkg
from autoregressive_speech_token_gb300 import sd as sdm

INVALID, UNSUPPORTED = -1, -7
P = 1 << 20          # a pointer-like number, 16-byte aligned: no accepted call is made with it


@pytest.fixture(scope="module", autouse=True)
def lib():
    from autoregressive_speech_token_gb300 import build
    build.build()
    return pkg.load_library()


def refused(code, words, fn, *a):
    with pytest.raises(pkg.SdError) as e:
        fn(*a)
    assert e.value.code == code and words in str(e.value), str(e.value)


def test_struct_sizes_match_the_header():
    assert C.sizeof(sdm.Pages) == 4 * 8 + 3 * 8 + 6 * 4
    assert C.sizeof(sdm.States) == 3 * 8 + 3 * 8 + 6 * 4
    assert C.sizeof(sdm.Rope) == 64 * 8 + 64 + 8


def _plan(**kw):
    d = dict(len=P, new=P, R=2, free=P, n_free=3, page=16, table=P, width=4, rows=5, total=P, start=P, slot=P, pos=P,
             req=P, info=P)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,words", [
    (dict(len=None), "NULL"), (dict(new=None), "NULL"), (dict(table=None), "NULL"), (dict(total=None), "NULL"),
    (dict(start=None), "NULL"), (dict(info=None), "NULL"), (dict(R=0), "R 0"), (dict(R=-3), "R -3"),
    (dict(n_free=-1), "n_free -1"), (dict(rows=-1), "rows -1"), (dict(width=0), "table_stride 0"),
    (dict(page=0), "page_size 0"), (dict(page=65537), "page_size 65537"), (dict(free=None), "free_dev"),
    (dict(slot=None), "slot_dev"), (dict(pos=None), "slot_dev"), (dict(req=None), "slot_dev"),
])
def test_plan_refusals(kw, words):
    refused(INVALID, words, pkg.sd_page_plan, *_plan(**kw))


def pages(**kw):
    d = dict(k_dev=P, v_dev=P, k_scale_dev=None, v_scale_dev=None, page_stride=0, head_stride=0, pos_stride=0,
             dtype=pkg.DTYPES["f16"], n_pages=4, page_size=16, n_kv_head=2, head_dim=64, reserved=0)
    d.update(kw)
    return sdm.Pages(*d.values())


BAD_PAGES = [
    (INVALID, dict(k_dev=None), "k_dev"), (INVALID, dict(v_dev=None), "v_dev"), (INVALID, dict(k_dev=P + 8), "aligned"),
    (INVALID, dict(dtype=1), "cache type 1"), (INVALID, dict(dtype=9), "cache type 9"),
    (UNSUPPORTED, dict(head_dim=96), "head_dim 96"), (INVALID, dict(n_pages=0), "0 pages"),
    (INVALID, dict(n_kv_head=0), "0 kv heads"), (INVALID, dict(page_size=0), "of 0 positions"),
    (INVALID, dict(page_size=65537), "of 65537"), (INVALID, dict(n_pages=1 << 20, page_size=1 << 12), "pages of"),
    (INVALID, dict(page_stride=4096, head_stride=1024, pos_stride=60), "multiples of 16"),
    (INVALID, dict(page_stride=-64, head_stride=64, pos_stride=64), "multiples of 16"),
    (INVALID, dict(k_scale_dev=P), "scales"),
]


def _write(rope="ok", cache=None, **kw):
    if rope == "ok":
        rope = pkg.sd_rope_init(64, 1e4)
    d = dict(pos=P, pos_stride=8, slot=P, n=8, dtype=pkg.DTYPES["f16"], q=P, q_stride=256, qo=P, qo_stride=256, H=4,
             k=P, v=P, kv_stride=128)
    d.update(kw)
    return [rope, *d.values(), cache if cache is not None else pages()]


@pytest.mark.parametrize("code,kw,words", BAD_PAGES)
def test_write_refuses_bad_caches(code, kw, words):
    refused(code, words, pkg.sd_rope_write_pages, *_write(cache=pages(**kw)))


@pytest.mark.parametrize("kw,words", [
    (dict(dtype=4), "type 4"), (dict(n=-1), "n -1"), (dict(slot=None), "NULL"), (dict(k=None), "NULL"),
    (dict(v=None), "NULL"), (dict(pos=None), "NULL"), (dict(q=None), "n_head > 0"), (dict(qo=None), "n_head > 0"),
    (dict(H=0), "n_head > 0"), (dict(q=P + 2), "16 bytes"), (dict(k=P + 4), "16 bytes"),
    (dict(kv_stride=129), "16 bytes"), (dict(q_stride=257), "16 bytes"), (dict(qo_stride=512), "another stride"),
    (dict(rope=sdm.Rope()), "head_dim"),
])
def test_write_refusals(kw, words):
    refused(INVALID, words, pkg.sd_rope_write_pages, *_write(**kw))


def test_write_refuses_another_heads_rope():
    refused(INVALID, "head_dim 128", pkg.sd_rope_write_pages, *_write(rope=pkg.sd_rope_init(128, 1e4)))


def test_calls_without_rows_do_nothing():
    pkg.sd_rope_write_pages(*_write(n=0, slot=None, pos=None, k=None, v=None))
    pkg.sd_attend_pages(*_attend(R=0, table=None, len=None, q=None, out=None))
    pkg.sd_attend_cross(*_cross(Lq=0, q=None, out=None))
    pkg.sd_attend_cross(*_cross(st=states(B=0, k_dev=None, v_dev=None), q=None, out=None))


@pytest.mark.parametrize("args,code,words", [
    ((96, 1e4), UNSUPPORTED, "head_dim"), ((64, 1.0), INVALID, "theta"), ((64, float("nan")), INVALID, "theta"),
    ((64, float("inf")), INVALID, "theta"), ((64, 1e4, [16, 15]), INVALID, "add up"),
    ((64, 1e4, [40, -8]), INVALID, "pairs[1]"), ((64, 1e4, [7, 7, 7, 7, 4]), INVALID, "5 axes"),
    ((64, 1e4, []), INVALID, "0 axes"),
])
def test_rope_init_refusals(args, code, words):
    refused(code, words, pkg.sd_rope_init, *args)


@pytest.mark.parametrize("hd,theta,pairs,inter", [
    (64, 1e4, None, False), (128, 1e6, None, False), (128, 1e6, [24, 20, 20], True), (128, 1e4, [16, 24, 24], False),
    (64, 5e5, [8, 8, 8, 8], True), (64, 1e4, [0, 32], True), (64, 1e4, [32, 0, 0], True)])
def test_rope_frequencies_and_axes(hd, theta, pairs, inter):
    r = pkg.sd_rope_init(hd, theta, pairs, inter)
    left, want, a = list(pairs or [hd // 2]), [], 0
    while len(want) < hd // 2:
        if left[a]:
            want.append(a)
            left[a] -= 1
            if not inter:
                continue
        a = (a + 1) % len(left)
    assert list(r.axis[:hd // 2]) == want and r.head_dim == hd and r.n_axes == len(left)
    turns = np.array([r.turn[i] for i in range(hd // 2)], np.float64) / 2.0 ** 64
    ref = theta ** (-2.0 * np.arange(hd // 2) / hd) / (2 * np.pi)
    # pow within 1 ulp, one division, one truncation at 2^-64 (far below a double's last bit of the smallest)
    assert np.all(np.abs(turns / ref - 1) < 4 * 2.0 ** -53 + 2.0 ** -64 / ref)


def _attend(cache=None, **kw):
    d = dict(ws=None, cache=cache if cache is not None else pages(), table=P, width=4, len=P, R=2,
             dtype=pkg.DTYPES["f16"], q=P, q_stride=256, H=4, scale=0.125, out=P, out_stride=256)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("code,kw,words", BAD_PAGES)
def test_attend_pages_refuses_bad_caches(code, kw, words):
    refused(code, words, pkg.sd_attend_pages, *_attend(cache=pages(**kw)))


@pytest.mark.parametrize("code,kw,words", [
    (INVALID, dict(table=None), "table_dev"), (INVALID, dict(len=None), "len_dev"), (INVALID, dict(width=0), "table_stride 0"),
    (INVALID, dict(R=-1), "R -1"), (INVALID, dict(dtype=4), "type 4"), (INVALID, dict(q=None), "q_dev"),
    (INVALID, dict(out=P + 8), "16 bytes"), (INVALID, dict(q_stride=250), "16 bytes"), (INVALID, dict(H=3), "n_head 3"),
    (INVALID, dict(H=0), "n_head 0"), (INVALID, dict(scale=float("inf")), "scale"),
    (INVALID, dict(scale=float("nan")), "scale"), (INVALID, dict(), "ws is NULL"),
    (UNSUPPORTED, dict(dtype=1, cache=pages(dtype=3)), "SD_F32 queries"),
    (UNSUPPORTED, dict(cache=pages(dtype=4, page_size=7)), "odd number"),
    (INVALID, dict(cache=pages(page_stride=0, head_stride=1024, pos_stride=64)), "positive"),
])
def test_attend_pages_refusals(code, kw, words):
    refused(code, words, pkg.sd_attend_pages, *_attend(**kw))


def states(**kw):
    d = dict(k_dev=P, v_dev=P, len_dev=None, batch_stride=0, head_stride=0, pos_stride=0, dtype=pkg.DTYPES["f16"], B=2,
             n_pos=10, n_kv_head=2, head_dim=64, reserved=0)
    d.update(kw)
    return sdm.States(*d.values())


def _cross(st=None, **kw):
    d = dict(ws=None, states=st if st is not None else states(), dtype=pkg.DTYPES["f16"], q=P, q_batch=1024,
             q_stride=256, Lq=4, H=4, scale=0.125, out=P, out_batch=1024, out_stride=256)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("code,st,kw,words", [
    (INVALID, dict(k_dev=None), {}, "k_dev"), (INVALID, dict(v_dev=P + 2), {}, "aligned"),
    (INVALID, dict(dtype=4), {}, "type 4"), (UNSUPPORTED, dict(head_dim=80), {}, "head_dim 80"),
    (INVALID, dict(B=-1), {}, "B -1"), (INVALID, dict(n_pos=-1), {}, "n_pos -1"), (INVALID, dict(n_kv_head=0), {}, "n_kv_head 0"),
    (INVALID, dict(batch_stride=1280, head_stride=64, pos_stride=132), {}, "strides"),
    (INVALID, dict(batch_stride=0, head_stride=64, pos_stride=128), {}, "positive"), (INVALID, {}, dict(Lq=-1), "Lq -1"), (INVALID, {}, dict(q_batch=1001), "q_batch"),
    (INVALID, {}, dict(out_batch=1001), "out_batch"), (INVALID, {}, dict(q_stride=100), "16 bytes"),
    (INVALID, {}, dict(H=5), "n_head 5"), (INVALID, {}, {}, "ws is NULL"),
    (UNSUPPORTED, dict(dtype=3), dict(dtype=1), "SD_F32 queries"),
])
def test_attend_cross_refusals(code, st, kw, words):
    refused(code, words, pkg.sd_attend_cross, *_cross(st=states(**st), **kw))


def test_null_structs(lib):
    assert lib.sd_attend_pages(None, None, P, 4, P, 2, 2, P, 256, 4, 0.1, P, 256, None, None) == INVALID
    assert lib.sd_attend_cross(None, None, 2, P, 0, 256, 1, 4, 0.1, P, 0, 256, None, None) == INVALID
    assert lib.sd_rope_write_pages(None, None, 0, P, 1, 2, None, 0, None, 0, 0, P, P, 128, None, None) == INVALID
    assert lib.sd_attn_ws_create(0, None) == INVALID
    assert lib.sd_rope_init(64, 1e4, 1, None, 0, None) == INVALID
    lib.sd_attn_ws_destroy(None)
