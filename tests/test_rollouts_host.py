"""Forked pages, shared prefixes and scores without a GPU: every refusal comes before
the first CUDA call."""

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


def _fork(**kw):
    d = dict(table=P, width=4, len=P, R=2, parent=P, N=3, free=P, n_free=5, page=16, n_pages=20, table_out=2 * P,
             len_out=P, copies=P, ref=P, free_out=P, info=P, work=P)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,words", [
    (dict(R=-1), "R -1"), (dict(N=-1), "N -1"), (dict(n_free=-2), "n_free -2"), (dict(width=0), "table_stride 0"),
    (dict(page=0), "page_size 0"), (dict(page=65537), "page_size 65537"), (dict(n_pages=0), "n_pages 0"),
    (dict(n_pages=2 ** 28), "n_pages"), (dict(table=None), "table_dev"), (dict(len=None), "len_dev"),
    (dict(parent=None), "parent_dev"), (dict(table_out=None), "table_out_dev"), (dict(len_out=None), "len_out_dev"),
    (dict(copies=None), "copy_dev"), (dict(free=None), "free_dev"), (dict(ref=None), "ref_dev"),
    (dict(free_out=None), "free_out_dev"), (dict(info=None), "info_dev"), (dict(work=None), "work_dev"),
    (dict(work=P + 4), "8-byte"), (dict(table_out=P), "table_out_dev is table_dev"),
])
def test_fork_refusals(kw, words):
    refused(INVALID, words, pkg.sd_page_fork, *_fork(**kw))


def _compact(**kw):
    d = dict(table=P, width=4, len=P, R=2, page=16, n_pages=20, table_out=P, copies=P, ref=P, free_out=P, info=P, work=P)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,words", [
    (dict(R=-1), "R -1"), (dict(width=0), "table_stride 0"), (dict(page=0), "page_size 0"), (dict(n_pages=0), "n_pages 0"),
    (dict(table=None), "table_dev"), (dict(len=None), "len_dev"), (dict(table_out=None), "table_out_dev"),
    (dict(copies=None), "copy_dev"), (dict(ref=None), "ref_dev"), (dict(free_out=None), "free_out_dev"),
    (dict(info=None), "info_dev"), (dict(work=None), "work_dev"), (dict(work=P + 4), "8-byte"),
])
def test_compact_refusals(kw, words):
    refused(INVALID, words, pkg.sd_page_compact, *_compact(**kw))


@pytest.mark.parametrize("kw,words", [
    (dict(width=2 ** 30 + 1), "table_stride 1073741825"), (dict(width=2 ** 31 - 1), "2^30"),
    (dict(page=1, n_pages=2 ** 26 + 1), "n_pages 67108865")])
def test_sizes_beyond_what_the_passes_count(kw, words):
    refused(UNSUPPORTED, words, pkg.sd_page_fork, *_fork(**kw))
    refused(UNSUPPORTED, words, pkg.sd_page_compact, *_compact(**kw))


def test_fork_of_too_many_rows():
    refused(UNSUPPORTED, "N 1048577", pkg.sd_page_fork, *_fork(N=2 ** 20 + 1))


def test_work_words():
    assert pkg.sd_page_work(-1, 0, 5) == 0 and pkg.sd_page_work(0, -1, 5) == 0 and pkg.sd_page_work(1, 1, 0) == 0
    assert pkg.sd_page_work(0, 0, 1) > 0
    # beyond 32 bits
    assert pkg.sd_page_work(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) > 2 ** 32 - 2


def pages(**kw):
    d = dict(k_dev=P, v_dev=P, k_scale_dev=None, v_scale_dev=None, page_stride=0, head_stride=0, pos_stride=0,
             dtype=pkg.DTYPES["f16"], n_pages=4, page_size=16, n_kv_head=2, head_dim=64, reserved=0)
    d.update(kw)
    return sdm.Pages(*d.values())


def test_copy_refusals():
    copy = pkg.sd_page_copy
    refused(INVALID, "n_caches 129", copy, [pages()] * 129, P, P, 3)
    refused(INVALID, "max_copies -1", copy, [pages()], P, P, -1)
    refused(INVALID, "NULL", copy, [pages()], None, P, 3)
    refused(INVALID, "NULL", copy, [pages()], P, None, 3)
    refused(UNSUPPORTED, "head_dim 96", copy, [pages(head_dim=96)], P, P, 3)
    refused(INVALID, "cache type", copy, [pages(dtype=pkg.DTYPES["f32"])], P, P, 3)
    for kw in (dict(dtype=pkg.DTYPES["bf16"]), dict(n_pages=5), dict(page_size=8), dict(n_kv_head=1), dict(head_dim=128),
               dict(page_stride=4096, head_stride=1024, pos_stride=64)):
        refused(INVALID, "cache 1", copy, [pages(), pages(**kw)], P, P, 3)
    copy([], P, P, 3)                                       # nothing to do
    copy([pages()], P, P, 0)


def _shared(**kw):
    d = dict(ws=P, cache=pages(), table=P, width=3, len=P, R=4, group=P, shared=P, n_groups=2, dtype=pkg.DTYPES["f16"], q=P,
             q_stride=256, H=4, scale=0.125, out=P, out_stride=256, lse=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("code,kw,words", [
    (INVALID, dict(n_groups=-1), "n_groups -1"), (INVALID, dict(n_groups=5), "n_groups 5"),
    (INVALID, dict(group=None), "group_dev"), (INVALID, dict(shared=None), "shared_dev"),
    (INVALID, dict(R=-1), "R -1"), (INVALID, dict(width=0), "table_stride 0"), (INVALID, dict(table=None), "table_dev"),
    (INVALID, dict(len=None), "len_dev"), (INVALID, dict(ws=None), "ws is NULL"), (INVALID, dict(q=P + 8), "16 bytes"),
    (INVALID, dict(H=3), "n_head 3"), (INVALID, dict(scale=float("nan")), "scale"),
    (INVALID, dict(dtype=pkg.DTYPES["e4m3"]), "type"),
    (UNSUPPORTED, dict(cache=pages(dtype=pkg.DTYPES["bf16"]), dtype=pkg.DTYPES["f32"]), "SD_F32"),
])
def test_shared_refusals(code, kw, words):
    refused(code, words, pkg.sd_attend_shared, *_shared(**kw))


def _score(**kw):
    d = dict(z=P, stride=100, dtype=pkg.DTYPES["f32"], rows=2, V=100, T=1.0, token=P, logp=P, rank=P, entropy=P, top=4,
             top_id=P, top_logp=P)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("code,kw,words", [
    (INVALID, dict(z=None), "logits_dev"), (INVALID, dict(z=P + 2), "aligned"), (INVALID, dict(rows=-1), "rows -1"),
    (INVALID, dict(V=0), "V 0"), (UNSUPPORTED, dict(V=262145, stride=262145), "V 262145"), (INVALID, dict(top=-1), "top_n -1"),
    (UNSUPPORTED, dict(top=33), "top_n 33"), (INVALID, dict(stride=99), "stride 99"), (INVALID, dict(T=0.0), "temperature"),
    (INVALID, dict(T=-1.0), "temperature"), (INVALID, dict(T=float("nan")), "temperature"),
    (INVALID, dict(T=float("inf")), "temperature"), (INVALID, dict(T=1e-31), "temperature"),
    (INVALID, dict(token=None), "token_dev"), (INVALID, dict(top_id=None), "top_id_dev"),
    (INVALID, dict(top_logp=None), "top_logp_dev"), (INVALID, dict(dtype=pkg.DTYPES["e4m3"]), "type"),
])
def test_score_refusals(code, kw, words):
    refused(code, words, pkg.sd_score_rows, *_score(**kw))


def test_calls_without_rows_do_nothing():
    pkg.sd_score_rows(*_score(rows=0, z=None))
    pkg.sd_attend_shared(*_shared(R=0, ws=None))
