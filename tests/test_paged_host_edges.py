"""Calls of the paged-cache and attention entries that a caller's loop can produce,
without a GPU."""

import pytest

import autoregressive_speech_token_gb300 as pkg
from autoregressive_speech_token_gb300 import sd as sdm

from .test_paged_host import _attend, _cross, _plan, _write, lib, pages, refused, states  # noqa: F401  (lib is a fixture)

INVALID = -1


@pytest.mark.parametrize("cache", [pages(k_dev=None, v_dev=None), pages(n_pages=0), None])
def test_no_rows_whatever_the_cache(cache):
    """An empty batch over a pool that is not there yet."""
    pkg.sd_rope_write_pages(None, None, 0, None, 0, pkg.DTYPES["f16"], None, 0, None, 0, 0, None, None, 0, cache)
    pkg.sd_attend_pages(None, cache, None, 0, None, 0, pkg.DTYPES["f16"], None, 0, 4, 0.1, None, 0)


@pytest.mark.parametrize("st", [states(k_dev=None, v_dev=None), states(B=0, k_dev=None, dtype=9), None])
def test_no_queries_whatever_the_states(st):
    Lq = 3 if st is not None and st.B == 0 else 0
    pkg.sd_attend_cross(None, st, pkg.DTYPES["f16"], None, 0, 0, Lq, 4, 0.1, None, 0, 0)


def test_a_plan_of_no_requests_is_refused():
    """It would still have start_dev[0], info_dev and the slots of `rows` tokens to write."""
    refused(INVALID, "R 0", pkg.sd_page_plan, *_plan(R=0))
