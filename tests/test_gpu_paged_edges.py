"""Paged and cross attention where a caller can be surprised: expired waits, large groups
of heads, scores of any size, queries of uneven elements."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from .test_gpu_paged import (DT, HALF_STEP, attend_ref, bounds, build_cache, check_cross, e4m3_values, gen, i32, make_states,  # noqa: E402
                             randn, run_cross, run_paged, sd, ws)  # noqa: F401  (sd and ws are fixtures)

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.mark.parametrize("kind,Lq,hd", [("pages", 1, 128), ("cross", 1, 64), ("cross", 300, 64), ("cross", 40, 128)])
def test_an_expired_wait_is_reported_and_replays_give_nan(sd, monkeypatch, kind, Lq, hd):  # noqa: F811
    """A test hook (SD_TEST_STALL_US) lets one load warp of the first uncaptured call wait 1 ms for a barrier that
    nothing arrives at; the other waits of its block end on the recorded error.  The next call with the workspace is
    refused.  A graph captured before has no host call that could refuse: its replays end and give NaN, not results
    that some units joined from records of another pass.  Another workspace works."""
    g = gen(50)
    lens = [3000, 900]
    monkeypatch.setenv("SD_TEST_STALL_US", "1000")
    w = sd.AttnWorkspace()
    monkeypatch.delenv("SD_TEST_STALL_US")
    good = sd.AttnWorkspace()
    ld = i32(lens)
    lse = torch.zeros(2, Lq, 4, device="cuda")
    if kind == "pages":
        kc, vc, table, _ = build_cache(g, np.random.default_rng(50), lens, 2, hd, 16, "f16", "hnd")
        q, cache = randn(g, 2, 4, hd, dt="f16"), sd.Pages.of(kc, vc)
        out = torch.zeros_like(q)

        def call(x):
            sd.sd_attend_pages(x, cache, table, table.shape[1], ld, 2, sd.DTYPES["f16"], q, 4 * hd, 4, 0.1, out, 4 * hd,
                               lse, torch.cuda.current_stream().cuda_stream)
    else:
        k, v = (randn(g, 2, 3000, 2, hd, dt="f16") for _ in range(2))
        q, states = randn(g, 2, Lq, 4, hd, dt="f16"), sd.States.of(k, v, ld)
        out = torch.zeros_like(q)

        def call(x):
            sd.sd_attend_cross(x, states, sd.DTYPES["f16"], q, q.stride(0), q.stride(1), Lq, 4, 0.1, out, q.stride(0),
                               q.stride(1), lse, torch.cuda.current_stream().cuda_stream)
    call(good)
    torch.cuda.synchronize()
    want, want_lse = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(w)                                                # captured: leaves the hook to the next call
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    call(w)                                                    # this one takes it
    torch.cuda.synchronize()
    for _ in range(2):
        with pytest.raises(sd.SdError) as e:
            call(w)
        assert e.value.code == TIMEOUT
    for _ in range(3):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.all(torch.isnan(out)) and torch.all(torch.isnan(lse))
    call(good)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def check_plain(q, k, v, lens, scale, out):
    """All heads against 64 bits; returns the share of elements that are the 64-bit result rounded once."""
    G, right = q.shape[2] // k.shape[2], []
    for b, n in enumerate(lens):
        kk, vv = (x[b, :n].double().repeat_interleave(G, 1) for x in (k, v))
        p = torch.softmax(torch.einsum("ihd,jhd->hij", q[b].double(), kk) * scale, -1)
        right.append(out[b] == torch.einsum("hij,jhd->ihd", p, vv).to(out.dtype))
    return torch.stack(right).double().mean().item()


@pytest.mark.parametrize("Lq,H,Hkv,hd,tiles", [
    (1, 64, 1, 64, False), (1, 64, 1, 128, False), (2, 64, 4, 128, False), (3, 16, 1, 128, False), (8, 64, 8, 64, False),
    (4, 40, 1, 64, False), (16, 16, 16, 128, False), (129, 4, 2, 64, True), (24, 8, 8, 128, True), (16, 64, 8, 128, True),
    (130, 64, 1, 64, True)])
def test_few_queries_of_large_groups_keep_fine_probabilities(sd, ws, Lq, H, Hkv, hd, tiles):  # noqa: F811
    """A tile of the tensor-core kernel holds queries of one head: with few queries to many heads nearly all of its
    rows are empty, and it rounds bf16 probabilities to 8 bits where the split kernel keeps 16.  400 probabilities of
    about 2^-8 rounding error each, averaged, move an element by about half of what rounding it moves it: a third or more of
    the elements round to a neighbour.  With 16 bits less than one in 20 does."""
    g = gen(51)
    lens, scale = [400, 250], hd ** -0.5
    k, v = make_states(g, lens, 400, Hkv, hd, "bf16", "blhd")
    q = randn(g, 2, Lq, H, hd, dt="bf16")
    out, lse = run_cross(sd, ws, q, k, v, lens, scale)
    check_cross(q, k, v, lens, scale, out, lse)
    share = check_plain(q, k, v, lens, scale, out)
    assert share < 0.75 if tiles else share > 0.95, share


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dt,kv,hd,Lq,e", [
    ("f16", "f16", 64, 3, 9), ("f16", "f16", 128, 8, 11), ("f32", "f16", 64, 8, 10), ("f32", "f16", 128, 2, 30),
    ("bf16", "f16", 64, 3, 11), ("bf16", "bf16", 128, 8, 40), ("f16", "f16", 64, 200, 9), ("f16", "f16", 128, 130, 11),
    ("f16", "f16", 64, 200, 15), ("f16", "f16", 128, 40, 13), ("bf16", "bf16", 64, 200, 10), ("bf16", "bf16", 128, 130, 40)])
def test_finite_scores_larger_than_their_steps(sd, ws, dt, kv, hd, Lq, e, sign):  # noqa: F811
    """Scores of 2^23 and more, where the step between fp32 numbers is 1 or more: a reference subtracted after rounding
    can be off by that many powers of two, beyond fp16's range.  One element of q and k is not 0, so the scores are
    exact; every seventh position ties for the largest, and the result is the mean of their values."""
    g = gen(52)
    n = 300
    q, k = torch.zeros(1, Lq, 1, hd, device="cuda"), torch.zeros(1, n, 1, hd, device="cuda")
    top = torch.arange(n, device="cuda") % 7 == 3
    q[0, :, 0, 5] = 2.0 ** e * (1 + torch.arange(Lq, device="cuda") % 8 / 8)
    k[0, :, 0, 5] = torch.where(top, 2.0 ** 14, 2.0 ** 13) if sign > 0 else torch.where(top, -2.0 ** 14, -2.0 ** 15)
    q, k, v = q.to(DT[dt]), k.to(DT[kv]), randn(g, 1, n, 1, hd, dt=kv)
    out, lse = run_cross(sd, ws, q, k, v, [n], 1.0)
    vt = v[0, top, 0].double()
    ref, mag = vt.mean(0).expand(Lq, hd), vt.abs().mean(0).expand(Lq, hd)
    tol, _ = bounds(ref, mag, torch.zeros(Lq, dtype=torch.float64, device="cuda"), n, dt, kv, hd)
    assert torch.all((out[0, :, 0].double() - ref).abs() <= tol)
    want = q[0, :, 0, 5].double() * sign * 2.0 ** 14
    assert torch.all((lse[0, :, 0].double() - want).abs() <= want.abs() * 2.0 ** -21)


@pytest.mark.parametrize("cache,hd", [("f16", 64), ("f16", 128), ("e4m3", 128), ("e4m3", 64)])
def test_fp32_queries_keep_their_bits_beside_a_large_element(sd, ws, cache, hd):  # noqa: F811
    """One element of a row is 2^12 times the others, whose keys are large while its own is small: the small elements
    make the scores, and an error relative to the row's largest would show."""
    g = gen(53)
    n, ps, H = 500, 16, 8
    big = 8.0 if cache == "f16" else 5.0
    kc, vc, table, rows = build_cache(g, np.random.default_rng(53), [n], 1, hd, ps, cache, "hnd")
    q = randn(g, 1, H, hd) * 2.0 ** -12
    q[..., 0] = 1.5
    k = rows[0][0].to(torch.float16).float() * 2.0 ** big
    k[..., 0] *= 2.0 ** -big * 2.0 ** -8
    k = k.clamp(-448, 448).to(DT[cache]) if cache == "e4m3" else k.to(DT[cache])
    slot = torch.arange(n, device="cuda")
    kc[table[0, slot // ps].long(), :, slot % ps] = k
    out, lse = run_paged(sd, ws, q, kc, vc, table, [n], 8.0)
    ref, mag, size, ls = attend_ref(q[0].double(), e4m3_values(k[:, 0]), e4m3_values(rows[0][1][:, 0]), 8.0)
    tol, tol_l = bounds(ref, mag, size, n, "f32", cache, hd)
    assert torch.all((out[0].double() - ref).abs() <= tol), float(((out[0].double() - ref).abs() / tol).max())
    assert torch.all((lse[0].double() - ls).abs() <= tol_l + ls.abs() * 2.0 ** -22)


def test_write_of_the_most_tokens(sd):  # noqa: F811
    """2^31 - 1 tokens, nearly all skipped, their rows one row of memory (stride 0)."""
    n, hd = 2 ** 31 - 1, 64
    slot = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slot[-1], slot[-4], slot[5] = 3, 9, 14
    x = randn(gen(54), 1, 2 * hd, dt="f16")
    kc, vc = (torch.zeros(1, 1, 16, hd, device="cuda", dtype=torch.float16) for _ in range(2))
    sd.sd_rope_write_pages(None, None, 0, slot, n, sd.DTYPES["f16"], None, 0, None, 0, 0, x, x[:, hd:], 0,
                           sd.Pages.of(kc, vc))
    torch.cuda.synchronize()
    used = torch.zeros(16, 1, dtype=torch.bool, device="cuda")
    used[[3, 9, 14]] = True
    assert torch.equal(kc[0, 0], torch.where(used, x[:, :hd], 0)) and torch.equal(vc[0, 0], torch.where(used, x[:, hd:], 0))


@pytest.mark.parametrize("dt,kv,Lq,H,Hkv,hd", [("f16", "f16", 32, 16, 16, 64), ("bf16", "bf16", 200, 4, 2, 128),
                                               ("f32", "f16", 32, 4, 4, 64), ("bf16", "bf16", 3, 8, 2, 128)])
@pytest.mark.parametrize("same", ["batch", "rows", "both"])
def test_queries_of_one_row_for_many(sd, ws, dt, kv, Lq, H, Hkv, hd, same):  # noqa: F811
    """Learned queries for every row of the batch, or one query repeated: strides of 0."""
    g = gen(55)
    lens = [300, 0, 141]
    k, v = make_states(g, lens, 300, Hkv, hd, kv, "blhd")
    q = randn(g, 1 if same != "rows" else 3, Lq if same == "batch" else 1, H, hd, dt=dt).expand(3, Lq, H, hd)
    out, lse = run_cross(sd, ws, q, k, v, lens, hd ** -0.5, pad=8)
    check_cross(q, k, v, lens, hd ** -0.5, out, lse)
    again, _ = run_cross(sd, ws, q.contiguous(), k, v, lens, hd ** -0.5)
    assert torch.equal(out, again)


def test_captured_calls_with_changed_lengths_against_plain(sd, ws):  # noqa: F811
    """All heads of a replayed paged and a replayed cross call against 64 bits, the lengths changed since the capture
    so that items are cut, left whole or empty."""
    g = gen(56)
    kc, vc, table, rows = build_cache(g, np.random.default_rng(56), [3000] * 4, 2, 128, 16, "f16", "hnd")
    q, cq = randn(g, 4, 8, 128, dt="f16"), randn(g, 4, 40, 8, 128, dt="f16")
    k, v = (randn(g, 4, 3000, 2, 128, dt="f16") for _ in range(2))
    ld, cache = i32([3000] * 4), sd.Pages.of(kc, vc)
    st = sd.States.of(k, v, ld)
    out, cout = torch.zeros_like(q), torch.zeros_like(cq)
    lse, clse = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 40, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream().cuda_stream
        sd.sd_attend_pages(ws, cache, table, table.shape[1], ld, 4, sd.DTYPES["f16"], q, 1024, 8, 0.1, out, 1024, lse, s)
        sd.sd_attend_cross(ws, st, sd.DTYPES["f16"], cq, 40 * 1024, 1024, 40, 8, 0.1, cout, 40 * 1024, 1024, clse, s)
    for n in ([3000, 5, 0, 700], [1, 2900, 64, 0], [0, 0, 0, 1], [1500] * 4, [128, 256, 257, 2999]):
        ld.copy_(i32(n))
        graph.replay()
        torch.cuda.synchronize()
        check_cross(cq, k, v, n, 0.1, cout, clse)
        pk, pv = (torch.stack([r[x] for r in rows]) for x in (0, 1))
        check_cross(q[:, None], pk, pv, n, 0.1, out[:, None], lse[:, None])


def test_many_short_rows_cut_or_whole_against_plain(sd, ws):  # noqa: F811
    """More rows than a warp's lanes with fewer items than SMs: parts are found by a walk over the rows."""
    g = gen(57)
    lens = [1500, 1, 0, 900] * 9
    k, v = make_states(g, lens, 1500, 1, 64, "bf16", "blhd")
    q = randn(g, len(lens), 30, 2, 64, dt="bf16")
    out, lse = run_cross(sd, ws, q, k, v, lens, 0.125)
    check_cross(q, k, v, lens, 0.125, out, lse)
