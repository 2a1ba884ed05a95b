"""Paged cache (tables, rotary write, attention) and cross attention against plain
64-bit implementations, at the sizes and masks where they can go wrong."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}


@pytest.fixture(scope="module")
def sd():
    import __graft_entry__
    __graft_entry__.build()
    import autoregressive_speech_token_gb300 as pkg
    assert torch.cuda.is_available()
    return pkg


@pytest.fixture(scope="module")
def ws(sd):
    w = sd.AttnWorkspace()
    yield w
    w.close()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dt="f32"):
    x = torch.randn(*shape, generator=g, device="cuda")
    return (x.half() if dt == "e4m3" else x).to(DT[dt])


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda").contiguous()


# ------------------------------------------------------------------ tables and slots

def plan_ref(ln, new, free, ps, table, rows):
    R, width = table.shape
    table = table.copy()
    slot, pos, req = [-1] * rows, [0] * rows, [-1] * rows
    start, total, used, bits, i = [], [], 0, 0, 0
    for r in range(R):
        start.append(i)
        if ln[r] < 0 or new[r] < 0:
            bits |= 8
        a, n = max(int(ln[r]), 0), max(int(new[r]), 0)
        total.append(a + n)
        old, every = -(-a // ps), -(-(a + n) // ps)
        if every > width:
            bits |= 4
        take = {}
        for p in range(old, min(every, width)):
            take[p] = int(free[used]) if used < len(free) else -1
            if i + p * ps - a < rows:
                table[r, p] = take[p]
            used += 1
        for x in range(a, min(a + n, a + max(rows - i, 0))):
            p = x // ps
            e = -1 if p >= width else take.get(p, int(table[r, p]) if p < old else -1)
            slot[i + x - a] = e * ps + x % ps if e >= 0 else -1
            pos[i + x - a], req[i + x - a] = x, r
        i += n
    bits |= (i > rows) | 2 * (used > len(free))
    return table, total, start + [i], slot, pos, req, [i, used, bits, max(total)]


def run_plan(sd, ln, new, free, ps, table, rows, stream=None):
    R, width = table.shape
    t = i32(table)
    out = dict(total=torch.full((R + 1,), -7, dtype=torch.int32, device="cuda"),
               start=torch.full((R + 2,), -7, dtype=torch.int32, device="cuda"),
               slot=torch.full((rows + 1,), -7, dtype=torch.int32, device="cuda"),
               pos=torch.full((rows + 1,), -7, dtype=torch.int32, device="cuda"),
               req=torch.full((rows + 1,), -7, dtype=torch.int32, device="cuda"),
               info=torch.full((5,), -7, dtype=torch.int32, device="cuda"))
    ld, nd, fd = i32(ln), i32(new), i32(free)
    for _ in range(2):                                     # the same call again changes nothing
        sd.sd_page_plan(ld, nd, R, fd if len(free) else None, len(free), ps, t, width, rows, out["total"],
                        out["start"], out["slot"], out["pos"], out["req"], out["info"], stream)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in out.items()}
    assert all(v[-1] == -7 for v in got.values())          # nothing behind the outputs
    return [t.cpu().numpy()] + [got[k][:-1] for k in ("total", "start", "slot", "pos", "req", "info")]


@pytest.mark.parametrize("R,ps,high,most,spare", [
    (1, 16, 40, 1, 3), (1, 1, 5, 9, 0), (16, 16, 425, 1, 29), (33, 7, 90, 40, 1), (513, 64, 3000, 3, 100),
    (1700, 32, 400, 5, 17), (3, 128, 1000, 2500, 5), (64, 65536, 70000, 900, 8), (5000, 16, 64, 2, 0)])
def test_plan_against_plain(sd, R, ps, high, most, spare):
    rng = np.random.default_rng(R * ps + most)
    ln = rng.integers(0, high, R)
    new = rng.integers(0, most + 1, R)
    ln[rng.random(R) < 0.2] = 0
    pages = -(-(ln + new) // ps)
    width = int(max(pages.max(), 1)) + 2
    ids = rng.permutation(int(pages.sum()) + 11)
    table = np.full((R, width), -1)
    at = 0
    for r in range(R):
        k = -(-int(ln[r]) // ps)
        table[r, :k] = ids[at:at + k]
        at += k
    rows = int(new.sum()) + spare
    want = plan_ref(ln, new, ids[at:], ps, table, rows)
    for g, w in zip(run_plan(sd, ln, new, ids[at:], ps, table, rows), want):
        np.testing.assert_array_equal(g, w)


@pytest.mark.parametrize("case", ["free", "rows", "wide", "negative", "nothing", "hole", "no_rows", "huge"])
def test_plan_when_things_run_out(sd, case):
    ln, new = np.array([5, 0, 31, 64, 12]), np.array([1, 40, 2, 1, 30])
    ps, width, rows = 16, 6, 80
    table = np.full((5, width), -1)
    for r in range(5):
        k = -(-int(ln[r]) // ps)
        table[r, :k] = 10 * r + np.arange(k)
    free = np.arange(100, 120)
    if case == "free":
        free = free[:3]
    elif case == "rows":
        rows = 37
    elif case == "wide":
        ln[3], new[3] = 90, 25
        table[3] = 30 + np.arange(width)
    elif case == "negative":
        ln[1], new[4] = -3, -9
    elif case == "nothing":
        new[:] = 0
    elif case == "hole":
        table[2, 1] = -1                                    # an entry lost earlier: its token has no slot
    elif case == "no_rows":
        rows = 0
    elif case == "huge":
        new[4] = 2 ** 31 - 1 - 12
        rows = 3000
    want = plan_ref(np.minimum(ln, 2 ** 31 - 1), new, free, ps, table, rows) if case != "huge" else None
    got = run_plan(sd, ln, new, free, ps, table, rows)
    if case == "huge":                                      # counts are limited, the table row ends the request
        assert got[1][4] == 2 ** 31 - 1 and got[2][5] == 2 ** 31 - 1 and got[6][2] & 5 == 5
        assert np.all(got[3][44 + 84:] == -1) and np.all(got[3][44:44 + 84] >= 0)
        return
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)


# ------------------------------------------------------------------ rotary write

def axis_of(hd, pairs, inter):
    left, out, a = list(pairs), [], 0
    while len(out) < hd // 2:
        if left[a]:
            out.append(a)
            left[a] -= 1
            if not inter:
                continue
        a = (a + 1) % len(left)
    return out


def turned(x, pos, axis, theta):
    """x [n][heads][hd] in 64 bits."""
    hd = x.shape[-1]
    f = theta ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64, device="cuda") / hd)
    ang = (pos.double()[axis].T * f)[:, None]
    a, b = x[..., :hd // 2], x[..., hd // 2:]
    return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)


def rounding(ref, mag, dt):
    """Half a step of the type (with its smallest numbers' step) plus fp32 rotation: a product, a fused sum and two
    factors good to 2 ulp on each element of the pair."""
    small = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0, "e4m3": 2.0 ** -10}[dt]
    return HALF_STEP[dt] * ref.abs() + small + mag * 8 * 2.0 ** -24


WRITES = [
    # n, H, Hkv, hd, dt, cache, ps, order, pairs, interleaved, theta, far
    (1, 16, 16, 64, "f32", "f16", 16, "hnd", [32], False, 1e4, 400),
    (16, 16, 8, 128, "f32", "f16", 16, "hnd", [64], False, 1e6, 425),
    (77, 16, 8, 128, "bf16", "bf16", 64, "nhd", [24, 20, 20], True, 1e6, 100000),
    (600, 6, 2, 64, "f16", "f16", 7, "pool", [8, 12, 12], False, 1e4, 2 ** 31 - 1),
    (513, 5, 1, 128, "bf16", "e4m3", 32, "hnd", [16, 16, 16, 16], True, 1e4, 5000),
    (33, 0, 4, 64, "f16", "e4m3", 1, "nhd", [32], False, 1e4, 5000),
    (40, 3, 3, 128, "f32", "bf16", 256, "hnd", [0, 64], True, 1e4, 5000),
    (9, 4, 4, 64, "f32", "e4m3", 8, "hnd", None, False, 1e4, 10),
]


def make_strides(order, n_pages, Hkv, ps, hd):
    if order == "nhd":
        return (ps * Hkv * hd, hd, Hkv * hd, 1)
    return ((3 if order == "pool" else 1) * Hkv * ps * hd, ps * hd, hd, 1)


def pool(order, n_pages, Hkv, ps, hd, dt, fill=7.0):
    """k and v in one order; "pool": every third block of a larger buffer."""
    st = make_strides(order, n_pages, Hkv, ps, hd)
    def one():
        size = sum((n - 1) * s for n, s in zip((n_pages, Hkv, ps, hd), st)) + 1
        flat = torch.full((size,), fill, device="cuda", dtype=torch.float16).to(DT[dt])
        return torch.as_strided(flat, (n_pages, Hkv, ps, hd), st)
    return one(), one()


@pytest.mark.parametrize("n,H,Hkv,hd,dt,cache,ps,order,pairs,inter,theta,far", WRITES)
@pytest.mark.parametrize("in_place", [False, True])
def test_write_against_plain(sd, n, H, Hkv, hd, dt, cache, ps, order, pairs, inter, theta, far, in_place):
    g = gen(n + hd)
    rng = np.random.default_rng(n)
    n_pages = -(-n // ps) + 3
    W = (H + 2 * Hkv) * hd + 16                             # rows of a fused projection, with a gap behind them
    x = randn(g, n, W, dt=dt)
    x0 = x.double()
    slot = rng.permutation(n_pages * ps)[:n]
    bad = rng.random(n) < 0.2
    slot = np.where(bad, rng.choice([-1, -5, n_pages * ps, 2 ** 31 - 1], n), slot)
    pos = i32(rng.integers(-far, far + 1, (len(pairs) if pairs else 1, n)))
    kc, vc = pool(order, n_pages, Hkv, ps, hd, cache)
    scales = (torch.rand(Hkv, generator=g, device="cuda") + 0.5, torch.rand(Hkv, generator=g, device="cuda") + 0.5) \
        if cache == "e4m3" else (None, None)
    qo = x if in_place else torch.full((n, H * hd + 16), 5.0, device="cuda", dtype=DT[dt])
    rope = sd.sd_rope_init(hd, theta, pairs, inter) if pairs else None
    q = x[:, :H * hd] if H else None
    sd.sd_rope_write_pages(rope, pos if pairs else None, n, i32(slot), n, sd.DTYPES[dt], q, W, qo if H else None,
                           qo.stride(0), H, x[:, H * hd:], x[:, (H + Hkv) * hd:], W, sd.Pages.of(kc, vc, *scales))
    torch.cuda.synchronize()
    ok = torch.as_tensor(~bad, device="cuda")
    s = torch.as_tensor(slot[~bad], device="cuda")
    axis = torch.as_tensor(axis_of(hd, pairs, inter), device="cuda") if pairs else None
    rot = (lambda y: turned(y, pos, axis, theta)) if pairs else (lambda y: y)
    mag = lambda y: (y.abs() + y.roll(hd // 2, -1).abs())
    if H:
        q0 = x0[:, :H * hd].reshape(n, H, hd)
        got = qo[:, :H * hd].double().reshape(n, H, hd)
        want = torch.where(ok[:, None, None], rot(q0), q0 if in_place else torch.full_like(q0, 5.0))
        assert torch.all((got - want).abs() <= rounding(want, mag(q0), dt) * ok[:, None, None])
        assert torch.all(qo[:, H * hd:(H * hd + 16)].double() == (x0[:, H * hd:H * hd + 16] if in_place else 5.0))
    for c, y, f, sc in ((kc, x0[:, H * hd:(H + Hkv) * hd], rot, scales[0]), (vc, x0[:, (H + Hkv) * hd:(H + 2 * Hkv) * hd],
                                                                            lambda y: y, scales[1])):
        y = y.reshape(n, Hkv, hd)
        inv = 1.0 if sc is None else 1.0 / sc.double()[None, :, None]
        want = torch.full((n_pages * ps, Hkv, hd), 7.0, device="cuda", dtype=torch.float64)
        tol = torch.zeros_like(want)
        want[s] = (f(y) * inv)[ok]
        tol[s] = rounding((f(y) * inv)[ok], (mag(y) * inv)[ok], cache)
        got = c.to(torch.float16 if cache == "e4m3" else c.dtype).double().transpose(1, 2).reshape(n_pages * ps, Hkv, hd)
        assert torch.all((got - want).abs() <= tol)


def test_write_saturates_and_keeps_nan(sd):
    k = torch.tensor([1e6, -1e6, float("nan"), float("inf"), 449.0, 0.0, -0.0, 1e-9] * 8, device="cuda").reshape(1, 64)
    kc, vc = pool("hnd", 1, 1, 1, 64, "e4m3", 0.0)
    sd.sd_rope_write_pages(None, None, 0, i32([0]), 1, sd.DTYPES["f32"], None, 0, None, 0, 0, k, k, 64,
                           sd.Pages.of(kc, vc))
    torch.cuda.synchronize()
    got = kc.float().reshape(8, 8)[0].tolist()
    assert got[0] == 448 and got[1] == -448 and math.isnan(got[2]) and got[3] == 448 and got[4] == 448
    assert got[5:] == [0, 0, 0]


# ------------------------------------------------------------------ attention

def attend_ref(q, k, v, scale):
    """q [M][hd], k / v [L][hd] in 64 bits: output, sum p|v|, largest sum |q k| scale, log-sum-exp."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device="cuda")
        return z, z, torch.zeros(q.shape[0], device="cuda", dtype=torch.float64), \
            torch.full((q.shape[0],), float("-inf"), device="cuda", dtype=torch.float64)
    s = q @ k.T * scale
    p = torch.softmax(s, -1)
    size = ((q.abs() @ k.abs().T) * abs(scale)).amax(-1)
    return p @ v, p @ v.abs(), size, torch.logsumexp(s, -1)


def bounds(ref, mag, size, n, dt, kv, hd):
    """|error| of an output element and of the log-sum-exp.
    Scores: q is held to 2^-22 (16-bit types: exact), hd products summed in fp32 with truncation, at most 2^-23 of
    the running sum each, hd/16 + 4 roundings deep; times `size`.  A score off by e moves a probability by e relative,
    and so does the denominator's share: 2 e.  exp2 and its argument: 2^-21 + 2^-23 * |score| (the argument's own
    rounding, |score| <= size).  Probabilities: 2^-22 relative for fp32 outputs; for 16-bit outputs rounded to the
    keys' and values' type.  Sums over n positions: at most n/16 + 64 roundings in sequence, 2^-23 each."""
    score = size * (2.0 ** -22 + (hd / 16 + 4) * 2.0 ** -23) + 2.0 ** -21 + size * 2.0 ** -23
    prob = 2.0 ** -22 if dt == "f32" else HALF_STEP["f16" if kv == "e4m3" else kv]
    sums = (n / 16 + 64) * 2.0 ** -23
    rel = (2 * score + prob + 2 * sums)[:, None]
    return mag * rel + HALF_STEP[dt] * (ref.abs() + mag * rel) + 1e-12, score + 2 * sums + 2.0 ** -20


def e4m3_values(x):
    return x.to(torch.float16).double() if x.dtype == torch.float8_e4m3fn else x.double()


def build_cache(g, rng, lens, Hkv, hd, ps, dt, order, holes=0.0):
    """Pages for the lengths in random order, NaN in every place that holds no position; the table has -1 and
    out-of-range ids behind each request's pages, and among them with `holes`."""
    held = [-(-n // ps) for n in lens]
    n_pages = sum(held) + 3
    ids = rng.permutation(n_pages)
    kc, vc = pool(order, n_pages, Hkv, ps, hd, dt, float("nan"))
    width = max(held + [1]) + 2
    table = rng.choice([-1, -9, n_pages, 2 ** 31 - 1], (len(lens), width))
    rows, at = [], 0
    for r, n in enumerate(lens):
        k, v = randn(g, n, Hkv, hd, dt=dt), randn(g, n, Hkv, hd, dt=dt)
        live = np.ones(n, bool)
        for p in range(held[r]):
            a, b = p * ps, min(n, p * ps + ps)
            if rng.random() < holes:
                live[a:b] = False
                continue
            table[r, p] = ids[at]
            kc[ids[at], :, :b - a] = k[a:b].transpose(0, 1)
            vc[ids[at], :, :b - a] = v[a:b].transpose(0, 1)
            at += 1
        live = torch.as_tensor(live, device="cuda")
        rows.append((k[live] if n else k, v[live] if n else v))
    return kc, vc, i32(table), rows


PAGED = [
    # lens, H, Hkv, hd, dt, cache, ps, order, holes
    ([1], 16, 16, 64, "f32", "f16", 16, "hnd", 0),
    ([399], 16, 16, 64, "f32", "f16", 16, "hnd", 0),
    ([0, 0], 4, 2, 128, "f16", "f16", 16, "hnd", 0),
    ([301, 302, 425, 17, 16, 15, 0, 1], 16, 8, 128, "f16", "f16", 16, "hnd", 0),
    ([1000, 3, 0, 64, 65, 63, 127, 128, 129], 6, 2, 64, "bf16", "bf16", 64, "nhd", 0),
    ([5000, 0, 1, 2500], 8, 1, 128, "bf16", "bf16", 128, "pool", 0),
    ([700, 11, 99], 12, 4, 128, "f16", "bf16", 7, "hnd", 0),
    ([513, 1024, 1], 16, 1, 64, "bf16", "f16", 1, "nhd", 0),
    ([2000, 41, 0, 333], 64, 8, 128, "bf16", "e4m3", 32, "hnd", 0),
    ([300, 299], 5, 1, 64, "f16", "e4m3", 8, "nhd", 0),
    ([90, 1234], 3, 3, 128, "f32", "e4m3", 48, "pool", 0),
    ([777], 40, 1, 128, "bf16", "bf16", 256, "hnd", 0),
    ([640, 200, 31], 8, 2, 64, "f16", "f16", 16, "hnd", 0.4),
    ([100, 320], 4, 4, 128, "bf16", "bf16", 5, "hnd", 0.3),
    ([33000], 8, 8, 64, "f32", "f16", 64, "hnd", 0),
    ([1, 2000, 0, 7] * 25, 8, 2, 128, "f16", "f16", 32, "nhd", 0),
    ([3000, 12], 4, 2, 128, "bf16", "e4m3", 512, "hnd", 0),
    ([900] * 3, 2, 1, 64, "bf16", "e4m3", 2, "hnd", 0.2),
    ([256, 512, 128, 384], 16, 16, 64, "f16", "f16", 1024, "hnd", 0),
    ([1300, 70], 9, 1, 128, "f32", "f16", 3, "pool", 0.1),
]


def run_paged(sd, ws, q, kc, vc, table, lens, scale, scales=(None, None), lse=True, stream=None):
    R, H, hd = q.shape
    out = torch.full((R + 1, H, hd), 9.0, device="cuda", dtype=q.dtype)
    ls = torch.full((R + 1, H), 9.0, device="cuda")
    sd.sd_attend_pages(ws, sd.Pages.of(kc, vc, *scales), table, table.shape[1], i32(lens), R, sd.dtype_of(q), q, H * hd,
                       H, scale, out, H * hd, ls if lse else None, stream)
    torch.cuda.synchronize()
    assert torch.all(out[R] == 9) and torch.all(ls[R] == 9)     # rows behind the last request
    return out[:R], ls[:R]


@pytest.mark.parametrize("lens,H,Hkv,hd,dt,cache,ps,order,holes", PAGED)
def test_paged_against_plain(sd, ws, lens, H, Hkv, hd, dt, cache, ps, order, holes):
    g, rng = gen(sum(lens) + H), np.random.default_rng(sum(lens))
    kc, vc, table, rows = build_cache(g, rng, lens, Hkv, hd, ps, cache, order, holes)
    q = randn(g, len(lens), H, hd, dt=dt)
    sc = (torch.rand(Hkv, generator=g, device="cuda") + 0.5, torch.rand(Hkv, generator=g, device="cuda") + 0.5) \
        if cache == "e4m3" else (None, None)
    scale = 1.0 / math.sqrt(hd)
    out, lse = run_paged(sd, ws, q, kc, vc, table, lens, scale, sc)
    again, _ = run_paged(sd, ws, q, kc, vc, table, lens, scale, sc, lse=False)
    assert torch.equal(out, again)
    G = H // Hkv
    for r, (k, v) in enumerate(rows):
        for kv in range(Hkv):
            kk, vv = e4m3_values(k[:, kv]), e4m3_values(v[:, kv])
            if sc[0] is not None:
                kk, vv = kk * sc[0][kv].double(), vv * sc[1][kv].double()
            ref, mag, size, ls = attend_ref(q[r, kv * G:(kv + 1) * G].double(), kk, vv, scale)
            tol, tol_l = bounds(ref, mag, size, k.shape[0], dt, cache, hd)
            assert torch.all((out[r, kv * G:(kv + 1) * G].double() - ref).abs() <= tol), (r, kv)
            d = lse[r, kv * G:(kv + 1) * G].double()
            assert torch.all((d == ls) | ((d - ls).abs() <= tol_l + ls.abs() * 2.0 ** -22)), (r, kv)


def test_paged_scores_far_apart(sd, ws):
    # one position outweighs the rest by e^60 in some rows; equal scores in others; all far below zero in others
    g = gen(5)
    n, hd, ps = 700, 64, 16
    kc, vc, table, rows = build_cache(g, np.random.default_rng(5), [n], 1, hd, ps, "f16", "hnd")
    q = torch.zeros(1, 3, hd, device="cuda")
    k, v = rows[0]
    q[0, 0] = k[311, 0].float() * 8
    q[0, 2, 0] = 1000.0
    out, _ = run_paged(sd, ws, q, kc, vc, table, [n], 1.0)
    ref, mag, size, _ = attend_ref(q[0].double(), k[:, 0].double(), v[:, 0].double(), 1.0)
    tol, _ = bounds(ref, mag, size, n, "f32", "f16", hd)
    assert torch.all((out[0].double() - ref).abs() <= tol)


def test_paged_large_queries_and_length_beyond_the_table(sd, ws):
    g = gen(6)
    kc, vc, table, rows = build_cache(g, np.random.default_rng(6), [64], 2, 64, 16, "f16", "hnd")
    table = table[:, :4].contiguous()
    q = randn(g, 1, 4, 64) * 1e7                              # above fp16's largest number
    out, _ = run_paged(sd, ws, q, kc, vc, table, [2 ** 31 - 1], 1e-7)
    for h in range(4):
        ref, mag, size, _ = attend_ref(q[0, h:h + 1].double(), rows[0][0][:, h // 2].double(),
                                       rows[0][1][:, h // 2].double(), 1e-7)
        tol, _ = bounds(ref, mag, size, 64, "f32", "f16", 64)
        assert torch.all((out[0, h:h + 1].double() - ref).abs() <= tol)
    zero, lse = run_paged(sd, ws, q, kc, vc, table, [-5], 1e-7)
    assert torch.all(zero == 0) and torch.all(lse == float("-inf"))


def test_paged_nan_of_a_used_position_reaches_its_rows_only(sd, ws):
    g = gen(7)
    kc, vc, table, _ = build_cache(g, np.random.default_rng(7), [40, 40], 2, 64, 16, "f16", "hnd")
    vc[table[1, 2].item(), 0, 3, 5] = float("nan")
    out, _ = run_paged(sd, ws, randn(g, 2, 4, 64, dt="f16"), kc, vc, table, [40, 40], 0.125)
    bad = torch.isnan(out)
    assert torch.all(bad[1, :2, 5]) and bad.sum() == 2


def test_paged_offsets_beyond_32_bits(sd, ws):
    # the last pages of a pool of more than 2^32 elements
    Hkv, ps, hd, n = 8, 64, 128, 150
    n_pages = 2 ** 32 // (Hkv * ps * hd) + 5
    g = gen(8)
    kc = torch.empty(n_pages, Hkv, ps, hd, device="cuda", dtype=torch.float8_e4m3fn)
    vc = torch.empty_like(kc)
    k, v = randn(g, n, Hkv, hd, dt="e4m3"), randn(g, n, Hkv, hd, dt="e4m3")
    ids = [n_pages - 1, n_pages - 4, n_pages - 2]
    slot = i32([ids[j // ps] * ps + j % ps for j in range(n)])
    cache = sd.Pages.of(kc, vc)
    sd.sd_rope_write_pages(None, None, 0, slot, n, sd.DTYPES["f32"], None, 0, None, 0, 0, k.float(), v.float(),
                           Hkv * hd, cache)
    q = randn(g, 1, 16, hd, dt="bf16")
    out, _ = run_paged(sd, ws, q, kc, vc, i32([ids]), [n], 0.09)
    for h in range(16):
        ref, mag, size, _ = attend_ref(q[0, h:h + 1].double(), e4m3_values(k[:, h // 2]), e4m3_values(v[:, h // 2]), 0.09)
        tol, _ = bounds(ref, mag, size, n, "bf16", "e4m3", hd)
        assert torch.all((out[0, h:h + 1].double() - ref).abs() <= tol)


@pytest.mark.parametrize("R", [3000, 70000])
def test_paged_many_requests(sd, ws, R):
    rng, g = np.random.default_rng(R), gen(R)
    hd, ps, n_pages = 64, 16, 500
    kc, vc = (randn(g, n_pages, 1, ps, hd, dt="f16") for _ in range(2))
    table = i32(rng.integers(0, n_pages, (R, 2)))
    lens = rng.integers(0, 33, R)
    q = randn(g, R, 1, hd, dt="f16")
    out, _ = run_paged(sd, ws, q, kc, vc, table, lens, 0.125)
    t = table.long()
    k = kc[t][:, :, 0].reshape(R, 2 * ps, hd).double()
    v = vc[t][:, :, 0].reshape(R, 2 * ps, hd).double()
    live = torch.arange(2 * ps, device="cuda")[None] < i32(lens)[:, None]
    s = torch.einsum("rd,rld->rl", q[:, 0].double(), k) * 0.125
    p = torch.softmax(s.masked_fill(~live, -1e30), -1) * live
    ref, mag = torch.einsum("rl,rld->rd", p, v), torch.einsum("rl,rld->rd", p, v.abs())
    size = torch.einsum("rd,rld->rl", q[:, 0].double().abs(), k.abs()).amax(-1) * 0.125
    tol, _ = bounds(ref, mag, size, 32, "f16", "f16", hd)
    assert torch.all((out[:, 0].double() - ref).abs() <= tol)


CROSS = [
    # lens, Lq, Lk, H, Hkv, hd, dt, kv, order
    ([150, 97], 32, 150, 16, 16, 64, "f32", "f16", "blhd"),
    ([1, 0, 7], 1, 7, 4, 4, 64, "f16", "f16", "blhd"),
    ([1500, 0, 801], 1, 1500, 16, 16, 64, "f16", "f16", "bhld"),
    ([300, 129], 3, 300, 16, 8, 128, "bf16", "bf16", "blhd"),
    ([257, 256, 255, 0], 130, 257, 4, 2, 128, "bf16", "bf16", "bhld"),
    ([1000], 777, 1000, 6, 2, 64, "f16", "f16", "blhd"),
    ([128, 127, 1], 256, 128, 5, 1, 64, "bf16", "bf16", "blhd"),
    ([700], 513, 700, 16, 1, 128, "f16", "f16", "blhd"),
    ([65], 1025, 65, 3, 3, 128, "bf16", "bf16", "bhld"),
    ([500, 3], 129, 500, 8, 8, 64, "f32", "f16", "bhld"),
    ([400, 77], 64, 400, 2, 2, 128, "f16", "bf16", "blhd"),
    ([400, 77], 200, 400, 4, 2, 64, "bf16", "f16", "blhd"),
    ([2049, 1], 300, 2049, 4, 4, 128, "f16", "f16", "blhd"),
    ([9001], 130, 9001, 2, 1, 128, "bf16", "bf16", "blhd"),
    ([4000, 0, 130, 1], 33, 4000, 4, 2, 64, "f16", "f16", "bhld"),
    ([300, 7, 0, 129, 1000] * 8, 20, 1000, 2, 2, 64, "bf16", "bf16", "blhd"),
    ([60, 0, 200] * 14, 3, 200, 12, 1, 128, "f16", "f16", "blhd"),
    ([900, 3], 17, 900, 1, 1, 64, "bf16", "bf16", "blhd"),
    ([1500, 1499], 16, 1500, 2, 2, 64, "f16", "f16", "blhd"),
]


def make_states(g, lens, Lk, Hkv, hd, kv, order):
    B = len(lens)
    def one():
        x = randn(g, B, Lk, Hkv, hd, dt=kv) if order == "blhd" else randn(g, B, Hkv, Lk, hd, dt=kv).transpose(1, 2)
        for b, n in enumerate(lens):
            x[b, n:] = float("nan")                            # what lies behind a length is not used
        return x
    return one(), one()


def run_cross(sd, ws, q, k, v, lens, scale, stream=None, lse=True, pad=0):
    B, Lq, H, hd = q.shape
    buf = torch.full((B, Lq + 1, H * hd + pad), 9.0, device="cuda", dtype=q.dtype)
    ls = torch.full((B * Lq * H + 1,), 9.0, device="cuda")
    length = i32(lens) if lens is not None else None
    sd.sd_attend_cross(ws, sd.States.of(k, v, length), sd.dtype_of(q), q, q.stride(0), q.stride(1), Lq, H, scale, buf,
                       buf.stride(0), buf.stride(1), ls if lse else None, stream)
    torch.cuda.synchronize()
    assert torch.all(buf[:, Lq] == 9) and torch.all(buf[:, :, H * hd:] == 9) and ls[-1] == 9
    return buf[:, :Lq, :H * hd].reshape(B, Lq, H, hd), ls[:-1].reshape(B, Lq, H)


def check_cross(q, k, v, lens, scale, out, lse):
    dt = {v: k for k, v in DT.items()}[q.dtype]
    kv = {v: k for k, v in DT.items()}[k.dtype]
    H, G, hd = q.shape[2], q.shape[2] // k.shape[2], q.shape[3]
    for b, n in enumerate(lens):
        for h in range(H):
            ref, mag, size, ls = attend_ref(q[b, :, h].double(), k[b, :n, h // G].double(), v[b, :n, h // G].double(), scale)
            tol, tol_l = bounds(ref, mag, size, n, dt, kv, hd)
            err = (out[b, :, h].double() - ref).abs()
            assert torch.all(err <= tol), (b, h, float((err / tol).max()))
            d = lse[b, :, h].double()
            assert torch.all((d == ls) | ((d - ls).abs() <= tol_l + ls.abs() * 2.0 ** -22)), (b, h)


@pytest.mark.parametrize("lens,Lq,Lk,H,Hkv,hd,dt,kv,order", CROSS)
def test_cross_against_plain(sd, ws, lens, Lq, Lk, H, Hkv, hd, dt, kv, order):
    g = gen(Lq + Lk + hd)
    k, v = make_states(g, lens, Lk, Hkv, hd, kv, order)
    q = randn(g, len(lens), Lq, H, hd, dt=dt)
    out, lse = run_cross(sd, ws, q, k, v, lens, 1 / math.sqrt(hd), pad=16)
    again, _ = run_cross(sd, ws, q, k, v, lens, 1 / math.sqrt(hd), lse=False)
    assert torch.equal(out, again)
    check_cross(q, k, v, lens, 1 / math.sqrt(hd), out, lse)


@pytest.mark.parametrize("Lq", [1, 200])
def test_cross_without_lengths_and_with_rows_of_a_projection(sd, ws, Lq):
    g = gen(31)
    B, Lk, H, hd = 2, 333, 4, 64
    qkv = randn(g, B, Lq, 3 * H * hd, dt="bf16")
    kv = randn(g, B, Lk, 2 * H * hd, dt="bf16")
    q = qkv[:, :, H * hd:2 * H * hd].unflatten(2, (H, hd))
    k, v = kv[:, :, :H * hd].unflatten(2, (H, hd)), kv[:, :, H * hd:].unflatten(2, (H, hd))
    out, lse = run_cross(sd, ws, q, k, v, None, 0.2)
    check_cross(q, k, v, [Lk] * B, 0.2, out, lse)


@pytest.mark.parametrize("Lq", [2, 300])
def test_cross_lengths_out_of_range_are_limited(sd, ws, Lq):
    g = gen(32)
    k, v = make_states(g, [70, 0], 70, 2, 128, "f16", "blhd")
    q = randn(g, 2, Lq, 4, 128, dt="f16")
    out, lse = run_cross(sd, ws, q, k, v, [2 ** 31 - 1, -2 ** 31], 0.1)
    check_cross(q, k, v, [70, 0], 0.1, out, lse)


@pytest.mark.parametrize("Lq,scale", [(1, -0.3), (150, -0.3), (1, 0.0), (150, 0.0), (4, 40.0), (260, 40.0)])
def test_cross_scales(sd, ws, Lq, scale):
    g = gen(33)
    k, v = make_states(g, [301], 301, 2, 64, "f16", "blhd")
    q = randn(g, 1, Lq, 2, 64, dt="f16")
    out, lse = run_cross(sd, ws, q, k, v, [301], scale)
    check_cross(q, k, v, [301], scale, out, lse)


@pytest.mark.parametrize("Lq", [1, 256])
def test_cross_infinite_scores(sd, ws, Lq):
    """A key of -inf-like scores takes no part; +inf gives NaN as the formula does; other queries are untouched."""
    g = gen(34)
    k, v = make_states(g, [200], 200, 1, 64, "f16", "blhd")
    k[0, 17, 0, :] = 0
    k[0, 17, 0, 0] = float("-inf")
    q = randn(g, 1, Lq, 1, 64, dt="f16").abs()
    out, lse = run_cross(sd, ws, q, k, v, [200], 0.125)
    keep = torch.arange(200, device="cuda") != 17
    check_cross(q, k[:, keep], v[:, keep], [199], 0.125, out, lse)
    k[0, 17, 0, 0] = float("inf")
    out, _ = run_cross(sd, ws, q, k, v, [200], 0.125)
    assert torch.all(torch.isnan(out))


# ------------------------------------------------------------------ together

def test_decode_steps_agree_with_the_contiguous_cache(sd, ws):
    """Prompts of four lengths, then 40 steps: tables, rotary write and attention from one captured graph, replayed;
    every step against sd_attend_rows over a contiguous copy of the same requests."""
    g = gen(40)
    R, H, Hkv, hd, ps, steps = 4, 16, 8, 128, 16, 40
    prompt = [37, 16, 0, 150]
    rope = sd.sd_rope_init(hd, 1e6)
    kc, vc = pool("hnd", 64, Hkv, ps, hd, "f16", float("nan"))
    cache = sd.Pages.of(kc, vc)
    width, rows = 16, 256
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    free = i32(np.random.default_rng(1).permutation(64))
    total, start, info = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (R, R + 1, 4))
    slot, pos, req = (torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(3))
    ln, new = i32([0] * R), i32(prompt)
    x = randn(g, rows, (H + 2 * Hkv) * hd)
    qo = torch.zeros(rows, H * hd, device="cuda")
    out = torch.zeros(R, H, hd, device="cuda")
    st = torch.cuda.Stream()

    def step(n, s, attend):
        sd.sd_page_plan(ln, new, R, free, free.numel(), ps, table, width, n, total, start, slot, pos, req, info, s)
        sd.sd_rope_write_pages(rope, pos, rows, slot, n, sd.DTYPES["f32"], x, x.stride(0), qo, H * hd, H,
                               x[:, H * hd:], x[:, (H + Hkv) * hd:], x.stride(0), cache, s)
        if attend:
            sd.sd_attend_pages(ws, cache, table, width, total, R, sd.DTYPES["f32"], qo, H * hd, H, hd ** -0.5, out,
                               H * hd, None, s)

    def take(used):
        ln.copy_(total)
        free.copy_(free.roll(-used))

    step(rows, None, False)                               # the prompts
    torch.cuda.synchronize()
    assert info.tolist()[:3] == [sum(prompt), sum(-(-n // ps) for n in prompt), 0]
    hist = [[], [], [], []]
    for i in range(sum(prompt)):
        hist[req[i].item()].append(slot[i].item())
    take(info[1].item())
    new.fill_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step(R + 2, torch.cuda.current_stream().cuda_stream, True)
    for i in range(steps):
        x.copy_(randn(g, *x.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert slot[R:R + 2].tolist() == [-1, -1] and info[2].item() == 0
        for r in range(R):
            hist[r].append(slot[r].item())
            n = len(hist[r])
            assert total[r].item() == n and pos[r].item() == n - 1 and req[r].item() == r
            s = torch.as_tensor(hist[r], device="cuda")
            k = kc.transpose(1, 2).reshape(-1, Hkv, hd)[s].transpose(0, 1).contiguous()
            v = vc.transpose(1, 2).reshape(-1, Hkv, hd)[s].transpose(0, 1).contiguous()
            want = torch.empty(1, H, hd, device="cuda")
            sd.sd_attend_rows(qo[r:r + 1], k, v, 1, H, Hkv, hd, n, n, 4, want)
            # both within the attention tests' 2e-5 of max |V|
            assert (out[r] - want[0]).abs().max() <= 4e-5 * v.abs().max()
        take(info[1].item())
    assert len({s for h in hist for s in h}) == sum(prompt) + R * steps


def test_two_streams_with_a_workspace_each(sd):
    g = gen(41)
    q = randn(g, 4, 8, 128, dt="bf16")
    lens = [3000, 2500, 0, 4000]
    kc, vc, table, _ = build_cache(g, np.random.default_rng(3), lens, 4, 128, 64, "bf16", "hnd")
    k, v = make_states(g, [1900, 700], 1900, 4, 128, "bf16", "blhd")
    cq = randn(g, 2, 200, 8, 128, dt="bf16")
    w = [sd.AttnWorkspace() for _ in range(2)]
    want_p, _ = run_paged(sd, w[0], q, kc, vc, table, lens, 0.1)
    want_c, _ = run_cross(sd, w[0], cq, k, v, [1900, 700], 0.1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    cache, states, ld = sd.Pages.of(kc, vc), sd.States.of(k, v, i32([1900, 700])), i32(lens)
    outs = [[torch.empty_like(q) for _ in range(20)], [torch.empty_like(cq) for _ in range(20)]]
    torch.cuda.synchronize()
    for i in range(20):
        sd.sd_attend_pages(w[0], cache, table, table.shape[1], ld, 4, sd.DTYPES["bf16"], q, 1024, 8, 0.1, outs[0][i],
                           1024, None, streams[0].cuda_stream)
        sd.sd_attend_cross(w[1], states, sd.DTYPES["bf16"], cq, 200 * 1024, 1024, 200, 8, 0.1, outs[1][i], 200 * 1024,
                           1024, None, streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want_p) for o in outs[0]) and all(torch.equal(o, want_c) for o in outs[1])


def test_two_graphs_share_a_workspace_in_turn(sd):
    g = gen(42)
    w = sd.AttnWorkspace()
    sets = []
    for lens in ([2000, 10], [900, 1800]):
        kc, vc, table, _ = build_cache(g, np.random.default_rng(4), lens, 2, 64, 16, "f16", "hnd")
        q = randn(g, 2, 4, 64, dt="f16")
        want, _ = run_paged(sd, w, q, kc, vc, table, lens, 0.125)
        out, ld, cache = torch.zeros_like(q), i32(lens), sd.Pages.of(kc, vc)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sd.sd_attend_pages(w, cache, table, table.shape[1], ld, 2, sd.DTYPES["f16"], q, 256, 4, 0.125, out, 256, None,
                               torch.cuda.current_stream().cuda_stream)
        sets.append((graph, out, want, (ld, cache, table, q)))
    for _ in range(5):
        for graph, out, want, _ in sets:
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_captured_calls_follow_their_lengths(sd, ws):
    """One capture of each attention call; the lengths change between the replays, and with them the shares."""
    g = gen(43)
    lens = [[3000, 5, 0, 700], [1, 2900, 64, 0], [0, 0, 0, 1], [1500, 1500, 1500, 1500]]
    full = [3000] * 4
    kc, vc, table, rows = build_cache(g, np.random.default_rng(9), full, 2, 128, 16, "f16", "hnd")
    q = randn(g, 4, 8, 128, dt="f16")
    k, v = (randn(g, 4, 3000, 2, 128, dt="f16") for _ in range(2))
    cq = randn(g, 4, 40, 8, 128, dt="f16")
    ld, cache = i32(full), sd.Pages.of(kc, vc)
    states = sd.States.of(k, v, ld)
    out, cout = torch.zeros_like(q), torch.zeros_like(cq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream().cuda_stream
        sd.sd_attend_pages(ws, cache, table, table.shape[1], ld, 4, sd.DTYPES["f16"], q, 1024, 8, 0.1, out, 1024, None, s)
        sd.sd_attend_cross(ws, states, sd.DTYPES["f16"], cq, 40 * 1024, 1024, 40, 8, 0.1, cout, 40 * 1024, 1024, None, s)
    for n in lens:
        ld.copy_(i32(n))
        graph.replay()
        torch.cuda.synchronize()
        a, _ = run_paged(sd, ws, q, kc, vc, table, n, 0.1)
        b, _ = run_cross(sd, ws, cq, k, v, n, 0.1)
        assert torch.equal(out, a) and torch.equal(cout, b)
        for r in range(4):
            kk, vv = rows[r][0][:n[r], 0].double(), rows[r][1][:n[r], 0].double()
            ref, mag, size, _ = attend_ref(q[r, :4].double(), kk, vv, 0.1)
            tol, _ = bounds(ref, mag, size, n[r], "f16", "f16", 128)
            assert torch.all((out[r, :4].double() - ref).abs() <= tol)


def test_one_page_pools_and_single_elements(sd, ws):
    """Dimensions of one element, whose strides mean nothing."""
    g = gen(44)
    kc, vc = randn(g, 1, 1, 1, 64, dt="f16"), randn(g, 1, 1, 1, 64, dt="f16")
    q = randn(g, 3, 1, 64, dt="f16")
    cache = sd.Pages.of(kc, vc)
    cache.page_stride = cache.head_stride = cache.pos_stride = 3
    out, ld = torch.zeros_like(q), i32([1, 0, 1])
    sd.sd_attend_pages(ws, cache, i32([[0], [0], [0]]), 1, ld, 3, sd.DTYPES["f16"], q, 64, 1, 0.1, out, 64)
    torch.cuda.synchronize()
    assert torch.equal(out[0], vc[0, 0]) and torch.equal(out[2], vc[0, 0]) and torch.all(out[1] == 0)


def test_workspace_of_the_device_and_calls_without_rows(sd, ws):
    kc, vc = pool("hnd", 2, 1, 16, 64, "f16", 0.0)
    cache = sd.Pages.of(kc, vc)
    q = torch.zeros(1, 1, 64, device="cuda", dtype=torch.float16)
    sd.sd_attend_pages(ws, cache, i32([[0]]), 1, i32([1]), 0, sd.DTYPES["f16"], q, 64, 1, 0.1, q, 64)
    st = sd.States.of(kc[:0].transpose(1, 2), vc[:0].transpose(1, 2))
    sd.sd_attend_cross(ws, st, sd.DTYPES["f16"], q, 64, 64, 1, 1, 0.1, q, 64, 64)
    # states without positions: zeros
    none = torch.zeros(2, 0, 1, 64, device="cuda", dtype=torch.float16)
    for Lq in (1, 40):
        cq = torch.ones(2, Lq, 2, 64, device="cuda", dtype=torch.float16)
        out = torch.full_like(cq, 5.0)
        sd.sd_attend_cross(ws, sd.States.of(none, none), sd.DTYPES["f16"], cq, Lq * 128, 128, Lq, 2, 0.1, out, Lq * 128, 128)
        torch.cuda.synchronize()
        assert torch.all(out == 0)
    with pytest.raises(sd.SdError):
        sd.AttnWorkspace(torch.cuda.device_count() + 7)
    w = sd.AttnWorkspace(0)
    w.close()
    w.close()
