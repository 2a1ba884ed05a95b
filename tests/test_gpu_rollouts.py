"""Forked, compacted and copied pages, attention with shared first pages, and scores of tokens against plain
implementations (64 bits where numbers are computed), at the sizes and masks where they can go wrong."""

import math

import numpy as np
import pytest

from tests.test_gpu_paged import attend_ref, bounds, e4m3_values, gen, i32, pool, randn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def sd():
    import __graft_entry__
    __graft_entry__.build()
    import autoregressive_speech_token_gb300 as pkg
    assert torch.cuda.is_available()
    return pkg


@pytest.fixture(scope="module", params=["always", "where_it_saves"])
def ws(sd, request):
    """Sharing whatever it saves, and by the library's own rule."""
    with pytest.MonkeyPatch.context() as m:
        if request.param == "always":
            m.setenv("SD_SHARE_MIN_BYTES", "0")
        w = sd.AttnWorkspace()
    yield w
    w.close()


# ------------------------------------------------------------------ fork

def clipped(n, ps, width):
    """(length as it counts, bits)."""
    bits = 8 * (n < 0)
    n = max(n, 0)
    if n > width * ps:
        return width * ps, bits | 4
    return n, bits


def fork_ref(table, ln, parent, free, ps, n_pages):
    R, width = table.shape
    lens, bits = [], 0
    for n in ln:
        x, b = clipped(int(n), ps, width)
        lens.append(x)
        bits |= b
    old = set()
    for r, n in enumerate(lens):
        for x in table[r, :-(-n // ps)].tolist():
            if 0 <= x < n_pages:
                old.add(x)
            else:
                bits |= 16
    out = np.full((len(parent), width), -1, np.int64)
    length, copies, seen, need = [], [], set(), 0
    for i, p in enumerate(parent):
        n = lens[p] if 0 <= p < R else 0
        k = -(-n // ps)
        if k:
            row = table[p, :k].astype(np.int64)
            out[i, :k] = np.where((row >= 0) & (row < n_pages), row, -1)
            if n % ps:
                if p in seen:
                    if need < len(free):
                        page = int(free[need])
                        if not 0 <= page < n_pages:
                            page = -1
                            bits |= 16
                        copies.append((out[i, k - 1], page, n % ps))
                    else:
                        page = -1
                        bits |= 2
                    need += 1
                    out[i, k - 1] = page
                    if page < 0:
                        n -= n % ps
                seen.add(p)
        length.append(n)
    ref = np.bincount(out[out >= 0], minlength=n_pages)[:n_pages]
    left = [int(x) for x in free[len(copies):]] + sorted(x for x in old if not ref[x])
    return out, length, copies, ref, left[:n_pages], [len(copies), min(len(left), n_pages), bits, max(length + [0])]


def run_fork(sd, table, ln, parent, free, ps, n_pages, stream=None):
    R, width = table.shape
    N = len(parent)
    new = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
    out, length, copies, ref = new(N + 1, width), new(N + 1), new(N + 1, 3), new(n_pages + 1)
    free_out, info, work = new(n_pages + 1), new(5), new(sd.sd_page_work(R, N, n_pages) + 1)
    t, n, p, f = i32(table), i32(ln), i32(parent), i32(free)
    for _ in range(2):                                     # the same call again changes nothing
        sd.sd_page_fork(t if R else None, width, n if R else None, R, p if N else None, N, f if len(free) else None,
                        len(free), ps, n_pages, out if N else None, length if N else None, copies if N else None, ref,
                        free_out, info, work, stream)
    torch.cuda.synchronize()
    assert work[-1] == -7
    return [x.cpu().numpy() for x in (out, length, copies, ref, free_out, info)]


def check_fork(sd, table, ln, parent, free, ps, n_pages):
    table, free = np.asarray(table).reshape(len(ln), -1), np.asarray(free, np.int64)
    want = fork_ref(table, ln, parent, free, ps, n_pages)
    out, length, copies, ref, free_out, info = run_fork(sd, table, ln, parent, free, ps, n_pages)
    N, c, left = len(parent), len(want[2]), len(want[4])
    np.testing.assert_array_equal(info, want[5] + [-7])
    np.testing.assert_array_equal(out[:N], want[0])
    np.testing.assert_array_equal(length[:N], want[1])
    np.testing.assert_array_equal(copies[:c], np.asarray(want[2]).reshape(-1, 3))
    np.testing.assert_array_equal(ref[:n_pages], want[3])
    np.testing.assert_array_equal(free_out[:left], want[4])
    # nothing behind the outputs
    assert (out[N] == -7).all() and length[N] == -7 and (copies[c:] == -7).all() and ref[-1] == -7
    assert (free_out[left:] == -7).all()
    return want


def rows_of(rng, lens, ps, spare, extra=2, beams=1):
    """Rows with pages in random order; groups of `beams` rows share the first half of their pages."""
    pages = [-(-n // ps) for n in lens]
    n_pages = sum(pages) + spare
    ids = rng.permutation(n_pages)
    table = rng.choice([-1, n_pages, 2 ** 31 - 1], (len(lens), max(pages + [1]) + extra))
    at = 0
    for r, k in enumerate(pages):
        if r % beams == 0:
            first = ids[at:at + (min(x for x in pages[r:r + beams]) // 2 if beams > 1 else 0)]
            at += len(first)
        table[r, :len(first)] = first
        own = k - len(first)
        table[r, len(first):k] = ids[at:at + own]
        at += own
    return table, ids[at:], n_pages


@pytest.mark.parametrize("lens,parent,ps,spare", [
    ([300], [0] * 16, 16, 20),                             # a prompt into rollouts
    ([300], [0] * 16, 16, 15),                             # exactly as many free pages as it takes
    ([304], [0] * 5, 16, 0),                               # full pages alone: nothing to copy
    ([1], [0, 0, 0], 64, 2), ([0], [0, 0], 8, 1), ([5], [-1], 8, 3), ([5, 9, 0], [2, 1, 0], 4, 0),
    ([7, 7, 7], [1, -1, 1, 3, 1, 2 ** 31 - 1, -2 ** 31], 7, 5),
    ([10, 20], [1, 1, 0, 0, 1], 1, 0), ([65536, 65537], [1, 1, 0], 65536, 4),
])
def test_fork_small(sd, lens, parent, ps, spare):
    table, free, n_pages = rows_of(np.random.default_rng(len(parent)), lens, ps, spare)
    check_fork(sd, table, lens, parent, free, ps, n_pages)


@pytest.mark.parametrize("R,N,ps,high,beams,spare", [
    (12, 50, 16, 400, 4, 60), (300, 1200, 16, 800, 4, 1500), (1000, 1000, 7, 300, 1, 9000), (2000, 2100, 64, 3000, 2, 70000),
    (64, 64, 1, 5000, 4, 10), (3, 9000, 32, 700, 1, 12000), (5000, 17, 16, 90, 1, 40), (40, 300, 8, 9000, 1, 200)])
def test_fork_against_plain(sd, R, N, ps, high, beams, spare):
    rng = np.random.default_rng(R + N)
    lens = np.repeat(rng.integers(0, high, R // beams), beams).tolist()
    parent = rng.integers(-R // 4, R + 1, N).tolist()
    table, free, n_pages = rows_of(rng, lens, ps, spare, beams=beams)
    check_fork(sd, table, lens, parent, free, ps, n_pages)


def test_fork_into_the_most_rows(sd):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, 1000).tolist()
    table, free, n_pages = rows_of(rng, lens, 16, 1 << 20)
    check_fork(sd, table, lens, rng.integers(-1, 1000, 1 << 20).tolist(), free, 16, n_pages)


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("case", ["short", "none", "wide", "negative", "bad_page", "bad_free", "no_new", "no_old", "nothing"])
def test_fork_when_things_go_wrong(sd, case, large):
    rng = np.random.default_rng(3)
    lens = [37, 64, 5, 90, 12] * (700 if large else 1)
    R, ps = len(lens), 16
    parent = [0, 0, 3, 3, 1, 4, 3, 2, 0] * (500 if large else 1)
    table, free, n_pages = rows_of(rng, lens, ps, 9000 if large else 9)
    if case == "short":
        free = free[:2]
    elif case == "none":
        free = free[:0]
    elif case == "wide":
        lens[3] = 2 ** 31 - 1
        table[3] = np.arange(table.shape[1])
    elif case == "negative":
        lens[0], lens[1] = -5, -2 ** 31
    elif case == "bad_page":
        table[0, 2], table[0, 0], table[1, 1] = n_pages, -2 ** 31, -1
    elif case == "bad_free":
        free[1], free[2] = -3, n_pages
    elif case == "no_new":
        parent = []
    elif case == "no_old":
        lens, table = [], np.zeros((0, 4), np.int64)
    elif case == "nothing":
        lens, table, parent, free = [], np.zeros((0, 4), np.int64), [], free[:0]
    check_fork(sd, table.reshape(len(lens), -1) if len(lens) else np.zeros((0, 4), np.int64), lens, parent, free, ps, n_pages) \
        if len(lens) else no_old_rows(sd, parent, free, ps, n_pages)


def no_old_rows(sd, parent, free, ps, n_pages):
    out, length, copies, ref, free_out, info = run_fork(sd, np.zeros((0, 4), np.int64), [], parent, free, ps, n_pages)
    N = len(parent)
    assert (out[:N] == -1).all() and (length[:N] == 0).all() and (ref[:n_pages] == 0).all()
    np.testing.assert_array_equal(free_out[:len(free)], free)
    np.testing.assert_array_equal(info, [0, len(free), 0, 0, -7])


def test_fork_again_and_again_keeps_every_page(sd):
    """Beams over many steps: the pages named and the free ones are all pages, each once, at every step."""
    rng = np.random.default_rng(11)
    ps, n_pages, width = 4, 400, 30
    table, lens, free = np.full((1, width), -1), [0], np.arange(n_pages)
    for step in range(40):
        parent = rng.integers(-1, len(lens), rng.integers(1, 9)).tolist()
        want = check_fork(sd, table, lens, parent, free, ps, n_pages)
        table, lens, free = want[0].copy(), list(want[1]), np.array(want[4])
        assert want[5][2] == 0
        for i, n in enumerate(lens):                       # a new token each
            if n % ps == 0:
                table[i, n // ps] = free[0]
                free = free[1:]
            lens[i] += 1
        named = set(table[table >= 0].tolist())
        assert not named & set(free.tolist()) and len(named) + len(free) == n_pages


@pytest.mark.parametrize("R,N", [(6, 20), (2500, 2400)])
def test_fork_and_compact_captured_and_on_two_streams(sd, R, N):
    """Two streams, a workspace each, replay a fork and a compaction of what it gave; the inputs change between the replays."""
    ps, n_pages, width = 8, 40000, 12
    new = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
    work = max(sd.sd_page_work(R, N, n_pages), sd.sd_page_work(N, 0, n_pages))
    sides = []
    for _ in range(2):
        x = dict(table=new(R, width), n=new(R), parent=new(N), free=new(30000), out=new(N, width), length=new(N), copies=new(N, 3),
                 ref=new(n_pages), free_out=new(n_pages), info=new(4), work=new(work), stream=torch.cuda.Stream(),
                 out2=new(N, width), moves=new(n_pages // 2, 3), ref2=new(n_pages), free2=new(n_pages), info2=new(4))
        torch.cuda.synchronize()
        x["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(x["graph"], stream=x["stream"]):
            s = x["stream"].cuda_stream
            sd.sd_page_fork(x["table"], width, x["n"], R, x["parent"], N, x["free"], 30000, ps, n_pages, x["out"], x["length"],
                            x["copies"], x["ref"], x["free_out"], x["info"], x["work"], s)
            sd.sd_page_compact(x["out"], width, x["length"], N, ps, n_pages, x["out2"], x["moves"], x["ref2"], x["free2"],
                               x["info2"], x["work"], s)
        sides.append(x)
    rng = np.random.default_rng(N)
    for _ in range(3):
        want = []
        for x in sides:
            lens = rng.integers(0, width * ps + 1, R)
            ids = rng.permutation(n_pages)
            table, free = ids[:10000][rng.integers(0, 10000, (R, width))], ids[10000:]
            parent = rng.integers(-1, R, N)
            want.append(fork_ref(table, lens.tolist(), parent.tolist(), free, ps, n_pages))
            for name, v in (("table", table), ("n", lens), ("parent", parent), ("free", free)):
                x[name].copy_(i32(v))
        torch.cuda.synchronize()
        for _ in range(3):
            for x in sides:
                with torch.cuda.stream(x["stream"]):
                    x["graph"].replay()
        torch.cuda.synchronize()
        for x, w in zip(sides, want):
            np.testing.assert_array_equal(x["info"].cpu(), w[5])
            np.testing.assert_array_equal(x["out"].cpu(), w[0])
            np.testing.assert_array_equal(x["length"].cpu(), w[1])
            np.testing.assert_array_equal(x["ref"].cpu(), w[3])
            np.testing.assert_array_equal(x["free_out"][:len(w[4])].cpu(), w[4])
            c = compact_ref(w[0], w[1], ps, n_pages)
            np.testing.assert_array_equal(x["info2"].cpu(), c[3])
            np.testing.assert_array_equal(x["out2"].cpu(), c[0])
            np.testing.assert_array_equal(x["moves"][:len(c[1])].cpu(), np.asarray(c[1]).reshape(-1, 3))


# ------------------------------------------------------------------ compact

def compact_ref(table, ln, ps, n_pages):
    R, width = table.shape
    bits, used = 0, np.zeros(table.shape, bool)
    for r, n in enumerate(ln):
        x, b = clipped(int(n), ps, width)
        bits |= b
        used[r, :-(-x // ps)] = True
    good = used & (table >= 0) & (table < n_pages)
    bits |= 16 * bool((used & ~good).any())
    live = sorted(set(table[good].tolist()))
    L = len(live)
    have = set(live)
    moves = list(zip([x for x in live if x >= L], [x for x in range(L) if x not in have]))
    to = np.arange(n_pages)
    for a, b in moves:
        to[a] = b
    out = np.where(good, to[np.where(good, table, 0)], -1)
    ref = np.bincount(out[out >= 0], minlength=n_pages)
    return out, [(a, b, ps) for a, b in moves], ref, [len(moves), n_pages - L, bits, L]


def check_compact(sd, table, ln, ps, n_pages):
    R, width = table.shape
    new = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
    out, copies, ref, free, info = new(R + 1, width), new(n_pages // 2 + 1, 3), new(n_pages + 1), new(n_pages + 1), new(5)
    work = new(sd.sd_page_work(R, 0, n_pages) + 1)
    for _ in range(2):
        sd.sd_page_compact(i32(table) if R else None, width, i32(ln) if R else None, R, ps, n_pages, out, copies, ref, free,
                           info, work)
    torch.cuda.synchronize()
    want = compact_ref(table, ln, ps, n_pages)
    got = [x.cpu().numpy() for x in (out, copies, ref, free, info)]
    m, L = want[3][0], want[3][3]
    np.testing.assert_array_equal(got[4], want[3] + [-7])
    np.testing.assert_array_equal(got[0][:R], want[0])
    np.testing.assert_array_equal(got[1][:m], np.asarray(want[1]).reshape(-1, 3))
    np.testing.assert_array_equal(got[2][:n_pages], want[2])
    np.testing.assert_array_equal(got[3][:n_pages - L], np.arange(L, n_pages))
    assert (got[0][R] == -7).all() and (got[1][m:] == -7).all() and got[2][-1] == -7 and work[-1] == -7
    assert (got[3][n_pages - L:] == -7).all()
    return want


@pytest.mark.parametrize("R,ps,high,beams,spare", [
    (1, 16, 100, 1, 0), (1, 16, 1, 1, 1), (3, 4, 50, 1, 64), (16, 16, 425, 4, 700), (600, 16, 700, 4, 100),
    (2000, 64, 5000, 1, 90000), (700, 1, 100, 1, 3), (5, 65536, 70000, 1, 31), (9000, 8, 20, 1, 5), (20, 16, 40000, 1, 33000)])
def test_compact_against_plain(sd, R, ps, high, beams, spare):
    rng = np.random.default_rng(R * ps)
    lens = np.repeat(rng.integers(0, high, -(-R // beams)), beams)[:R].tolist()
    table, _, n_pages = rows_of(rng, lens, ps, spare, beams=beams)
    check_compact(sd, table, lens, ps, max(n_pages, 1))


def test_compact_the_largest_pool(sd):
    rng = np.random.default_rng(9)
    n_pages = 1 << 26
    table = rng.integers(0, n_pages, (300, 7))
    table[0, :3] = 0, n_pages - 1, 2000
    check_compact(sd, table, rng.integers(0, 7 * 16 + 1, 300).tolist(), 16, n_pages)


@pytest.mark.parametrize("n_pages", [40, 20000])
def test_compact_when_things_go_wrong(sd, n_pages):
    table = np.arange(24).reshape(4, 6) % 21 + n_pages - 21
    check_compact(sd, table, [-1, 1000, 17, 0], 16, n_pages)        # negative and too long
    table[1, 1], table[2, 0] = n_pages, -9
    check_compact(sd, table, [96, 96, 96, 96], 16, n_pages)         # page ids that there are not
    check_compact(sd, table, [0, 0, 0, 0], 16, n_pages)             # nothing in use
    check_compact(sd, np.zeros((0, 3), np.int64), [], 16, n_pages)
    full = np.arange(n_pages)[::-1].reshape(1, -1).copy()
    check_compact(sd, full, [n_pages * 16], 16, n_pages)            # everything in use


# ------------------------------------------------------------------ copy

@pytest.mark.parametrize("copies,layers,Hkv,ps,hd,dt,order", [
    (1, 1, 1, 1, 64, "e4m3", "hnd"), (15, 28, 8, 16, 128, "f16", "hnd"), (7, 3, 5, 7, 64, "bf16", "nhd"),
    (300, 2, 2, 64, 128, "e4m3", "pool"), (33, 128, 1, 16, 64, "f16", "nhd"), (64, 1, 16, 256, 64, "bf16", "hnd"),
    (2, 1, 3, 65536, 64, "e4m3", "hnd"), (500, 4, 4, 1, 128, "f16", "pool")])
def test_copy_against_plain(sd, copies, layers, Hkv, ps, hd, dt, order):
    g, rng = gen(copies + layers), np.random.default_rng(copies)
    n_pages = 2 * copies + 3
    ids = rng.permutation(n_pages)
    pairs = np.stack([ids[:copies], ids[copies:2 * copies], rng.integers(0, ps + 2, copies)], 1)   # 0 and more than a page too
    pairs[:1, 2] = ps
    extra = [[ids[-1], n_pages, 1], [-1, ids[-2], 1], [ids[-3], ids[-3], ps], [ids[-1], ids[-2], ps]]   # the last is behind the count
    raw = lambda x: x.view(torch.uint8) if dt == "e4m3" else x
    k, v = ([pool(order, n_pages, Hkv, ps, hd, dt)[0] for _ in range(layers)] for _ in range(2))
    for x in k + v:
        x.copy_(randn(g, n_pages, Hkv, ps, hd, dt=dt))
    want = [[raw(x).clone() for x in y] for y in (k, v)]
    caches = [sd.Pages.of(a, b) for a, b in zip(k, v)]
    sd.sd_page_copy(caches, i32(np.concatenate([pairs, extra])), i32([copies + 3]), copies + 4)
    torch.cuda.synchronize()
    for pools, mine in zip((k, v), want):
        for x, w in zip(pools, mine):
            for a, b, n in pairs.tolist():
                w[b, :, :min(n, ps)] = w[a, :, :min(n, ps)]
            assert torch.equal(raw(x), w)
    # no more than max_copies, none for a negative count
    sd.sd_page_copy(caches, i32(np.concatenate([pairs[:0], extra[3:]])), i32([5]), 0)
    sd.sd_page_copy(caches, i32(np.concatenate([pairs[:0], extra[3:]])), i32([-5]), 1)
    torch.cuda.synchronize()
    assert all(torch.equal(raw(x), w) for pools, mine in zip((k, v), want) for x, w in zip(pools, mine))


def test_copy_offsets_beyond_32_bits(sd):
    Hkv, ps, hd = 8, 64, 128
    n_pages = 2 ** 32 // (Hkv * ps * hd) + 5
    k = torch.empty(n_pages, Hkv, ps, hd, device="cuda", dtype=torch.float8_e4m3fn)
    v = torch.empty_like(k)
    x = randn(gen(1), 2, Hkv, ps, hd, dt="e4m3").view(torch.uint8)
    k.view(torch.uint8)[3], v.view(torch.uint8)[n_pages - 1] = x[0], x[1]
    sd.sd_page_copy([sd.Pages.of(k, v)], i32([[3, n_pages - 2, ps], [n_pages - 1, 5, ps]]), i32([2]), 2)
    torch.cuda.synchronize()
    assert torch.equal(k.view(torch.uint8)[n_pages - 2], x[0]) and torch.equal(v.view(torch.uint8)[5], x[1])


# ------------------------------------------------------------------ shared first pages

def build_groups(g, rng, groups, loose, Hkv, hd, ps, dt, order, holes=0.0):
    """groups: (pages in common, lengths); loose: lengths behind them.  NaN where no position is."""
    width = max([-(-n // ps) for _, ls in groups for n in ls] + [-(-n // ps) for n in loose] + [s for s, _ in groups] + [1]) + 2
    n_pages = sum(s + sum(max(-(-n // ps) - s, 0) for n in ls) for s, ls in groups) + sum(-(-n // ps) for n in loose) + 3
    ids = rng.permutation(n_pages).tolist()
    kc, vc = pool(order, n_pages, Hkv, ps, hd, dt, float("nan"))
    table, rows, lens, at = [], [], [], 0

    def page(a, b):
        """A page with positions [a, b): its id (-1: a hole), keys and values."""
        nonlocal at
        k, v = randn(g, b - a, Hkv, hd, dt=dt), randn(g, b - a, Hkv, hd, dt=dt)
        if rng.random() < holes:
            return -1, k[:0], v[:0]
        i, at = ids[at], at + 1
        kc[i, :, :b - a] = k.transpose(0, 1)
        vc[i, :, :b - a] = v.transpose(0, 1)
        return i, k, v

    for s, ls in groups + [(0, [n]) for n in loose]:
        common = [page(0, min(ps, max(max(ls) - p * ps, 1))) for p in range(s)]
        for n in ls:
            row, ks, vs = rng.choice([-1, n_pages, 2 ** 31 - 1], width), [], []
            for p in range(max(-(-n // ps), 0)):
                m = min(ps, n - p * ps)
                i, k, v = common[p] if p < s else page(0, m)
                row[p] = i
                ks.append(k[:m])
                vs.append(v[:m])
            row[:s] = [c[0] for c in common]               # the same pages, whatever the length
            z = randn(g, 0, Hkv, hd, dt=dt)
            rows.append((torch.cat([raw16(x) for x in ks + [z]]), torch.cat([raw16(x) for x in vs + [z]])))
            table.append(row)
            lens.append(n)
    starts = np.cumsum([0] + [len(ls) for _, ls in groups])
    return kc, vc, i32(np.array(table)), rows, lens, i32(starts), i32([s for s, _ in groups])


def raw16(x):
    return x.half() if x.dtype == torch.float8_e4m3fn else x


def run_shared(sd, ws, q, cache, table, lens, starts, shared, scale, stream=None, lse=True):
    R, H, hd = q.shape
    out = torch.full((R + 1, H, hd), 9.0, device="cuda", dtype=q.dtype)
    ls = torch.full((R + 1, H), 9.0, device="cuda")
    sd.sd_attend_shared(ws, cache, table, table.shape[1], lens if torch.is_tensor(lens) else i32(lens), R, starts, shared,
                        shared.numel(), sd.dtype_of(q), q, H * hd, H, scale, out, H * hd, ls if lse else None, stream)
    torch.cuda.synchronize()
    assert torch.all(out[R] == 9) and torch.all(ls[R] == 9)
    return out[:R], ls[:R]


def check_rows(q, rows, out, lse, Hkv, scale, dt, cache, sc=(None, None)):
    G, hd = q.shape[1] // Hkv, q.shape[2]
    for r, (k, v) in enumerate(rows):
        for kv in range(Hkv):
            kk, vv = k[:, kv].double(), v[:, kv].double()
            if sc[0] is not None:
                kk, vv = kk * sc[0][kv].double(), vv * sc[1][kv].double()
            h = slice(kv * G, (kv + 1) * G)
            ref, mag, size, ls = attend_ref(q[r, h].double(), kk, vv, scale)
            tol, tol_l = bounds(ref, mag, size, k.shape[0], dt, cache, hd)
            good = bool(torch.all((out[r, h].double() - ref).abs() <= tol))
            assert good, (r, kv, (out[r, h].double() - ref).abs().max().item())
            d = lse[r, h].double()
            good = bool(torch.all((d == ls) | ((d - ls).abs() <= tol_l + ls.abs() * 2.0 ** -22)))
            assert good, (r, kv, d.tolist(), ls.tolist())


SHARED = [
    # groups of (pages in common, lengths), loose lengths, H, Hkv, hd, dt, cache, ps, order, holes
    ([(18, list(range(301, 317)))], [], 16, 8, 128, "f16", "f16", 16, "hnd", 0),
    ([(18, [300] * 16)], [], 16, 16, 64, "f32", "f16", 16, "hnd", 0),
    ([(70, [4500 + 7 * i for i in range(9)])], [33, 0], 8, 2, 128, "bf16", "bf16", 64, "nhd", 0),
    ([(40, [2600 + i for i in range(40)]), (3, [200, 210]), (0, [5, 700]), (50, [3200])], [1], 8, 2, 64, "f16", "f16", 64, "hnd", 0),
    ([(100, [1600 + i for i in range(70)])], [], 16, 4, 64, "f32", "f16", 16, "pool", 0),
    ([(9, [0, 5, 600, 576, 575, 577, 100, 64])], [10], 4, 4, 64, "bf16", "bf16", 64, "hnd", 0),   # shorter than what is shared
    ([(30, [2100 + i for i in range(33)])], [], 64, 8, 128, "bf16", "bf16", 64, "hnd", 0),
    ([(200, [1800, 1407, 1500, 1400])] * 3, [], 12, 4, 128, "f16", "f16", 7, "hnd", 0),
    ([(12, [3100 + i for i in range(20)])], [17], 16, 1, 64, "bf16", "bf16", 256, "hnd", 0),
    ([(33, [2200 + i for i in range(130)])], [], 4, 1, 128, "f16", "f16", 64, "hnd", 0),            # 520 rows to a kv head
    ([(500, [510, 511, 600])], [2], 8, 2, 64, "f16", "f16", 1, "nhd", 0),
    ([(2, [2100, 2048, 2500, 3000])], [], 16, 8, 128, "bf16", "bf16", 1024, "hnd", 0),
    ([(60, [2000 + i for i in range(24)])], [], 64, 8, 128, "bf16", "e4m3", 32, "hnd", 0),
    ([(40, [1400 + i for i in range(8)])], [], 4, 2, 64, "f32", "e4m3", 32, "hnd", 0),
    ([(20, [1500 + i for i in range(8)])], [], 8, 4, 128, "f16", "bf16", 64, "hnd", 0),
    ([(20, [1500 + i for i in range(8)])], [], 8, 4, 128, "bf16", "f16", 64, "hnd", 0),
    ([(60, [1000 + i for i in range(30)])], [400], 8, 2, 128, "f16", "f16", 16, "hnd", 0.3),
    ([(60, [1000 + i for i in range(30)])], [400], 8, 2, 64, "f32", "f16", 16, "hnd", 0.6),
    ([(64, [1030 + i for i in range(2)])] * 40, [900] * 9, 8, 2, 64, "bf16", "bf16", 16, "hnd", 0),
]


@pytest.mark.parametrize("groups,loose,H,Hkv,hd,dt,cache,ps,order,holes", SHARED)
def test_shared_against_plain(sd, ws, groups, loose, H, Hkv, hd, dt, cache, ps, order, holes):
    g, rng = gen(H * ps + len(groups)), np.random.default_rng(ps + hd)
    kc, vc, table, rows, lens, starts, shared = build_groups(g, rng, groups, loose, Hkv, hd, ps, cache, order, holes)
    q = randn(g, len(lens), H, hd, dt=dt)
    sc = tuple(torch.rand(Hkv, generator=g, device="cuda") + 0.5 for _ in range(2)) if cache == "e4m3" else (None, None)
    scale = 1.0 / math.sqrt(hd)
    pages = sd.Pages.of(kc, vc, *sc)
    out, lse = run_shared(sd, ws, q, pages, table, lens, starts, shared, scale)
    again, _ = run_shared(sd, ws, q, pages, table, lens, starts, shared, scale, lse=False)
    assert torch.equal(out, again)
    check_rows(q, rows, out, lse, Hkv, scale, dt, cache, sc)


@pytest.mark.parametrize("dt,scale", [("f16", -0.2), ("f16", 0.0), ("f16", 30.0), ("f32", -0.2), ("f32", 0.0), ("f32", 30.0),
                                      ("bf16", 1e-3)])
def test_shared_scales(sd, ws, dt, scale):
    g = gen(3)
    cache = "bf16" if dt == "bf16" else "f16"
    kc, vc, table, rows, lens, starts, shared = build_groups(g, np.random.default_rng(2), [(80, [1300 + i for i in range(12)])],
                                                             [], 2, 64, 16, cache, "hnd")
    q = randn(g, 12, 8, 64, dt=dt)
    out, lse = run_shared(sd, ws, q, sd.Pages.of(kc, vc), table, lens, starts, shared, scale)
    check_rows(q, rows, out, lse, 2, scale, dt, cache)


def test_shared_scores_far_apart(sd, ws):
    # one position of the prefix, or of the own part, outweighs the rest; rows with large queries; scores beyond fp16
    g = gen(5)
    kc, vc, table, rows, lens, starts, shared = build_groups(g, np.random.default_rng(5), [(60, [1000 + i for i in range(10)])],
                                                             [], 1, 64, 16, "f16", "hnd")
    for dt in ("f32", "f16"):
        q = torch.zeros(10, 2, 64, device="cuda")
        q[0, 0] = rows[0][0][311, 0].float() * 8
        q[1, 1] = rows[1][0][990, 0].float() * 8
        q[2, 0, 0] = 1000.0
        q[3, 0] = rows[3][0][959, 0].float() * 8
        if dt == "f32":
            q[4] = 1e6
        q = q.to(DT[dt])
        out, lse = run_shared(sd, ws, q, sd.Pages.of(kc, vc), table, lens, starts, shared, 1.0)
        check_rows(q, rows, out, lse, 1, 1.0, dt, "f16")


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_shared_values_that_are_not_finite(sd, ws, dt):
    g = gen(7)
    kc, vc, table, rows, lens, starts, shared = build_groups(g, np.random.default_rng(7), [(80, [1300 + i for i in range(4)])],
                                                             [1300], 2, 64, 16, "f16", "hnd")
    vc[table[1, 2].item(), 0, 3, 5] = float("nan")          # a page in common
    vc[table[2, 80].item(), 1, 3, 9] = float("inf")         # one of its own
    q = randn(g, 5, 4, 64, dt=dt)
    out, _ = run_shared(sd, ws, q, sd.Pages.of(kc, vc), table, lens, starts, shared, 0.125)
    bad = ~torch.isfinite(out)
    assert torch.all(bad[:4, :2, 5]) and torch.all(bad[2, 2:, 9]) and bad.sum() == 4 * 2 + 2
    if dt == "f32":
        return
    # scores of -inf alone: zeros
    kc[:] = torch.where(torch.isnan(kc), kc, torch.full_like(kc, float("-inf")))
    q = torch.zeros(5, 4, 64, device="cuda", dtype=DT[dt])
    q[..., 0] = 1
    for p in range(80):
        kc[table[0, p].item(), ..., 1:] = 0
    for r in range(5):
        for p in range(80 if r < 4 else 0, 82):
            kc[table[r, p].item(), ..., 1:] = 0
    vc[:] = torch.nan_to_num(vc, 0.0, 0.0, 0.0)
    out, lse = run_shared(sd, ws, q, sd.Pages.of(kc, vc), table, lens, starts, shared, 0.125)
    assert torch.all(out == 0) and torch.all(lse == float("-inf"))


def test_shared_groups_out_of_range_are_limited(sd, ws):
    g = gen(9)
    kc, vc, table, rows, lens, starts, shared = build_groups(g, np.random.default_rng(9), [(70, [1200 + i for i in range(6)])],
                                                             [1000], 2, 64, 16, "f16", "hnd")
    q = randn(g, 7, 4, 64, dt="f16")
    pages = sd.Pages.of(kc, vc)
    # more pages than a row has entries, bounds outside the requests, empty and negative groups
    for s, n in (([0, 6], [70]), ([-5, 0, 6, 6, 99], [3, 70, 9, -1]), ([0, 1, 6, 7], [10 ** 9, 60, -7]), ([6, 7], [5]),
                 ([4, 2, 6], [70, 70]), ([0, 0], [70])):
        out, lse = run_shared(sd, ws, q, pages, table, lens, i32(s), i32(n), 0.125)
        check_rows(q, rows, out, lse, 2, 0.125, "f16", "f16")


def test_shared_with_strides_streams_and_graphs(sd, monkeypatch):
    monkeypatch.setenv("SD_SHARE_MIN_BYTES", "0")
    g = gen(10)
    spec = [(64, [1100 + 3 * i for i in range(16)]), (40, [900, 700])]
    kc, vc, table, rows, lens, starts, shared = build_groups(g, np.random.default_rng(1), spec, [50], 4, 128, 16, "bf16", "hnd")
    R, H, hd = len(lens), 8, 128
    qkv = randn(g, R, 3 * H, hd, dt="bf16")                 # rows of a fused projection
    q = qkv[:, H:2 * H].contiguous()
    pages, ld = sd.Pages.of(kc, vc), i32(lens)
    w = [sd.AttnWorkspace() for _ in range(2)]
    want, _ = run_shared(sd, w[0], q, pages, table, ld, starts, shared, 0.1)
    out = torch.zeros(R, 2 * H, hd, device="cuda", dtype=torch.bfloat16)
    call = lambda ws, o, s: sd.sd_attend_shared(ws, pages, table, table.shape[1], ld, R, starts, shared, 2, sd.DTYPES["bf16"],
                                                qkv.data_ptr() + H * hd * 2, 3 * H * hd, H, 0.1, o, 2 * H * hd, None, s)
    call(w[0], out, None)
    torch.cuda.synchronize()
    assert torch.equal(out[:, :H], want) and torch.all(out[:, H:] == 0)
    # two streams at once, a workspace each
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [[torch.zeros_like(out) for _ in range(10)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(10):
        for s in range(2):
            call(w[s], outs[s][i], streams[s].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o[:, :H], want) for x in outs for o in x)
    # captured: lengths, groups and prefixes are read at every replay
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(w[0], out, torch.cuda.current_stream().cuda_stream)
    for ls, ss in ((lens, [64, 40]), ([x - 30 for x in lens], [64, 20]), (lens, [0, 40]), ([0] * R, [64, 40])):
        ld.copy_(i32(ls))
        shared.copy_(i32(ss))
        graph.replay()
        torch.cuda.synchronize()
        check_rows(q, [(k[:max(n, 0)], v[:max(n, 0)]) for (k, v), n in zip(rows, ls)], out[:, :H],
                   run_shared(sd, w[1], q, pages, table, ls, starts, shared, 0.1)[1], 4, 0.1, "bf16", "bf16")


def test_shared_many_requests(sd, ws):
    # more rows than the workspace has room for partial results
    g, rng = gen(12), np.random.default_rng(12)
    R, H, Hkv, hd, ps = 9000, 8, 8, 64, 16
    kc, vc = (randn(g, 400, Hkv, ps, hd, dt="f16") for _ in range(2))
    table = i32(np.concatenate([np.tile(rng.permutation(400)[:80], (R, 1)), rng.integers(0, 400, (R, 2))], 1))
    lens = rng.integers(1280, 1312, R)
    q = randn(g, R, H, hd, dt="f16")
    out, lse = run_shared(sd, ws, q, sd.Pages.of(kc, vc), table, lens, i32([0, R]), i32([80]), 0.125)
    for r in (0, 1, 4500, R - 1):
        ids = table[r].long()
        k, v = (x[ids].transpose(1, 2).reshape(-1, Hkv, hd)[:lens[r]] for x in (kc, vc))
        check_rows(q[r:r + 1], [(k, v)], out[r:r + 1], lse[r:r + 1], Hkv, 0.125, "f16", "f16")
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("hd,dt", [(128, "f16"), (64, "f32")])
def test_shared_expired_wait_is_reported_and_replays_give_nan(sd, monkeypatch, hd, dt):
    """A test hook (SD_TEST_STALL_US) lets a load warp of the first uncaptured call wait 1 ms for a barrier that nothing
    arrives at.  The next call with the workspace is refused; replays of a graph captured before give NaN; another
    workspace works."""
    g = gen(14)
    kc, vc, table, rows, lens, starts, shared = build_groups(g, np.random.default_rng(14), [(60, [970 + 9 * i for i in range(12)])],
                                                             [200], 2, hd, 16, "f16", "hnd")
    q, cache, ld = randn(g, 13, 4, hd, dt=dt), sd.Pages.of(kc, vc), i32(lens)
    monkeypatch.setenv("SD_SHARE_MIN_BYTES", "0")
    good = sd.AttnWorkspace()
    monkeypatch.setenv("SD_TEST_STALL_US", "1000")
    w = sd.AttnWorkspace()
    monkeypatch.delenv("SD_TEST_STALL_US")
    out, lse = torch.zeros_like(q), torch.zeros(13, 4, device="cuda")

    def call(x):
        sd.sd_attend_shared(x, cache, table, table.shape[1], ld, 13, starts, shared, 1, sd.DTYPES[dt], q, 4 * hd, 4, 0.1, out,
                            4 * hd, lse, torch.cuda.current_stream().cuda_stream)

    call(good)
    torch.cuda.synchronize()
    want, want_lse = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(w)                                            # captured: leaves the hook to the next call
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    call(w)                                                # this one takes it
    torch.cuda.synchronize()
    for _ in range(2):
        with pytest.raises(sd.SdError) as e:
            call(w)
        assert e.value.code == -6
    for _ in range(3):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.all(torch.isnan(out)) and torch.all(torch.isnan(lse))
    call(good)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


# ------------------------------------------------------------------ scores

def score_ref(z, T, token, top):
    """64 bits, from the definition."""
    V = z.numel()
    x = z.double().cpu().numpy()
    T = float(np.float32(T))
    live = x > -np.inf
    if not live.any():
        lp, H = np.full(V, -np.inf), 0.0
    else:
        d = (x - x.max()) / T
        lp = d - np.log(np.exp(d).sum())
        p = np.exp(lp)
        H = -(p[p > 0] * lp[p > 0]).sum()
    order = np.lexsort((np.arange(V), -x))
    order = order[live[order]][:top]
    ids = np.full(top, -1)
    ids[:len(order)] = order
    lps = np.full(top, -np.inf)
    lps[:len(order)] = lp[order]
    if 0 <= token < V:
        rank = int((x > x[token]).sum() + (x[:token] == x[token]).sum())
        return lp[token], rank, H, ids, lps
    return 0.0, -1, H, ids, lps


def run_score(sd, z, T, token, top, stream=None):
    rows, V = z.shape
    f = lambda *s: torch.full(s, 9.0, device="cuda")
    i = lambda *s: torch.full(s, 9, dtype=torch.int32, device="cuda")
    logp, rank, H, ids, lps = f(rows + 1), i(rows + 1), f(rows + 1), i(rows + 1, top), f(rows + 1, top)
    sd.sd_score_rows(z, z.stride(0), sd.dtype_of(z), rows, V, T, i32(token), logp, rank, H, top, ids if top else None,
                     lps if top else None, stream)
    torch.cuda.synchronize()
    for x in (logp, rank, H, ids, lps):
        assert torch.all(x[rows] == 9)
    return [x[:rows].cpu().numpy() for x in (logp, rank, H, ids, lps)]


def near(a, b):
    """log p within its roundings.  S has up to 64 terms a thread, then 5 + 16 + 5 additions, 2^-24 each, and exp2's and its
    argument's 2^-21 in all: below 128 * 2^-24 relative, an absolute error of log S.  (z - m) / T has two roundings, the
    difference with log S one, log one: 4 * 2^-24 of |log p| and of log S, at most log V < 13."""
    if b < -3.4028235e38:                                   # beyond fp32
        return np.isneginf(a)
    return abs(a - b) <= 128 * 2.0 ** -24 + 4 * 2.0 ** -24 * (2 * abs(b) + 13)


def check_score(sd, z, T, token, top):
    got = run_score(sd, z, T, token, top)
    again = run_score(sd, z, T, token, top)
    assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got, again))
    for r in range(z.shape[0]):
        lp, rank, H, ids, lps = score_ref(z[r], T, int(token[r]), top)
        assert near(got[0][r], lp), (r, got[0][r], lp)
        assert got[1][r] == rank, r
        # both terms are sums over the same terms: twice log S's bound, and a relative one of D / S
        assert abs(got[2][r] - H) <= 256 * 2.0 ** -24 + 256 * 2.0 ** -24 * H, (r, got[2][r], H)
        np.testing.assert_array_equal(got[3][r], ids)
        assert all(near(a, b) for a, b in zip(got[4][r], lps)), r


@pytest.mark.parametrize("rows,V,dt,T,top", [
    (1, 1, "f32", 1.0, 1), (3, 2, "f16", 0.7, 5), (2, 7, "bf16", 1.0, 32), (16, 2048, "f32", 0.9, 5), (400, 6563, "f32", 0.8, 20),
    (33, 8194, "f32", 0.8, 32), (700, 1025, "f16", 1.0, 3), (700, 4099, "bf16", 1.3, 8), (1, 131075, "bf16", 1.0, 8),
    (5, 50257, "f16", 0.5, 16), (2, 262144, "f32", 1.0, 32), (3, 262144, "f16", 1.0, 1), (150, 70001, "bf16", 1.0, 0),
    (1000, 33, "f32", 2.0, 32), (1, 20000, "f32", 1.0, 0)])
@pytest.mark.parametrize("lead,pad", [(0, 0), (3, 1), (1, 7)])
def test_score_against_plain(sd, rows, V, dt, T, top, lead, pad):
    g = gen(rows + V)
    flat = torch.full((rows * (V + pad) + lead,), 100.0, device="cuda", dtype=DT[dt])       # what is not the rows' would win
    z = flat[lead:].view(rows, V + pad)[:, :V]
    z.copy_(randn(g, rows, V) * 3)
    token = np.random.default_rng(V).integers(-1, V, rows)
    check_score(sd, z, T, token, top)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 60000])
def test_score_ties_order_and_masks(sd, V, dt):
    lowest = torch.finfo(DT[dt]).min
    z = torch.zeros(12, V, device="cuda", dtype=DT[dt])
    up = torch.linspace(-20, 20, V, device="cuda")
    z[1] = up.to(z.dtype)                                    # sorted up, then down: one block's threads hold all of the first
    z[2] = up.flip(0).to(z.dtype)
    z[3] = float("-inf")                                     # masked but for three
    z[3, [V // 2, 1, V - 1]] = 1.0
    z[4] = lowest                                            # masked with the lowest value, all alike
    z[5] = lowest
    z[5, V // 3] = 0.0
    z[6, ::2] = -0.0                                         # both zeros are alike
    z[7] = -(2.0 ** 12)                                      # far from zero, close together
    z[7, V // 2:] -= 8.0
    z[8] = lowest
    z[8, V - 2] = -lowest                                    # from the lowest to the largest
    z[9] = float("-inf")
    z[9, 7] = lowest
    z[10, ::3] = float("-inf")
    z[11] = torch.arange(V, device="cuda") % 5 - 2.0
    token = np.array([V - 1, V // 2, 3, 1, V // 2, V // 3, 1, V - 1, V - 2, 7, 1, V - 3])
    check_score(sd, z, 1.0, token, 32)
    check_score(sd, z, 0.7, (token + 1) % V, 1)


def test_score_a_sorted_row_with_many_entries_above_the_bound(sd):
    # the largest entries all with the threads of few groups: more reach the bound than the list holds
    for dt, V, threads, per in (("f32", 12000, 512, 4), ("bf16", 24000, 512, 8), ("f16", 8000, 128, 8)):
        rows = 1 if threads == 512 else 700
        z = randn(gen(V), rows, V, dt=dt)
        owner = (torch.arange(V, device="cuda") // per) % threads // 4
        for r in range(min(rows, 2)):
            z[r, owner < 32] += 50
        token = np.full(rows, 11)
        got = run_score(sd, z, 1.0, token, 32)
        for r in range(min(rows, 3)):
            _, rank, _, ids, _ = score_ref(z[r], 1.0, 11, 32)
            assert got[1][r] == rank
            np.testing.assert_array_equal(got[3][r], ids)


@pytest.mark.parametrize("V,dt,top", [(131075, "f32", 32), (262144, "f32", 9), (262141, "bf16", 32), (140001, "f16", 1)])
def test_score_long_rows_of_one_block(sd, V, dt, top):
    """Rows enough that none is cut: the bound of what is put aside rises while a row passes."""
    rows = 160
    z = randn(gen(V), rows, V, dt=dt) * 2
    up = torch.linspace(-9, 9, V, device="cuda")
    z[0] = up.to(z.dtype)                                    # every round above the one before
    z[1] = up.flip(0).to(z.dtype)
    z[2] = 0.5                                               # all alike
    z[3] = float("-inf")                                     # nothing in the first round but one
    z[3, 17] = -3.0
    z[3, V // 2 + 100:V // 2 + 160] = up[:60].to(z.dtype)
    z[4] = torch.finfo(DT[dt]).min
    z[5, :V // 8] -= 40                                      # the best behind the first eighth of each quarter
    token = np.random.default_rng(V).integers(0, V, rows)
    got, again = run_score(sd, z, 1.1, token, top), run_score(sd, z, 1.1, token, top)
    assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got, again))
    # S: V / 1024 terms in each half of a thread's pair, 32 additions behind, exp2 and its argument as in `near`
    tol = (V / 1024 + 96) * 2.0 ** -24
    ok = lambda a, b: np.isneginf(a) if b < -3.4028235e38 else abs(a - b) <= tol + 4 * 2.0 ** -24 * (2 * abs(b) + 13)
    for r in (*range(7), 80, rows - 1):
        lp, rank, H, ids, lps = score_ref(z[r], 1.1, int(token[r]), top)
        assert ok(got[0][r], lp) and got[1][r] == rank, r
        assert abs(got[2][r] - H) <= 2 * tol * (1 + H), r
        np.testing.assert_array_equal(got[3][r], ids)
        assert all(ok(a, b) for a, b in zip(got[4][r], lps)), r


@pytest.mark.parametrize("V", [100, 60000])
def test_score_rows_without_a_distribution(sd, V):
    z = torch.zeros(4, V, device="cuda")
    z[0] = float("-inf")
    z[1, 50] = float("nan")
    z[2, 60] = float("inf")
    logp, rank, H, ids, lps = run_score(sd, z, 1.0, [3, 3, 60, 3], 4)
    assert np.isneginf(logp[0]) and H[0] == 0 and (ids[0] == -1).all() and np.isneginf(lps[0]).all() and rank[0] == 3
    assert np.isnan(logp[1]) and np.isnan(H[1]) and np.isnan(lps[1]).all() and ids[1].tolist() == [0, 1, 2, 3] and rank[1] == 3
    assert np.isnan(logp[2]) and np.isnan(H[2]) and np.isnan(lps[2]).all() and ids[2].tolist() == [60, 0, 1, 2] and rank[2] == 0
    assert near(logp[3], -math.log(V))


def test_score_optional_outputs_streams_and_graphs(sd):
    z = randn(gen(4), 20, 5000, dt="bf16")
    token = i32(np.arange(20))
    f = lambda *s: torch.zeros(s, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    want = run_score(sd, z, 0.9, np.arange(20), 6)
    H, ids, lps, logp, rank = f(20), i(20, 6), f(20, 6), f(20), i(20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sd.sd_score_rows(z, 5000, sd.DTYPES["bf16"], 20, 5000, 0.9, None, None, None, H, stream=side.cuda_stream)
    sd.sd_score_rows(z, 5000, sd.DTYPES["bf16"], 20, 5000, 0.9, None, None, None, None, 6, ids, lps, side.cuda_stream)
    sd.sd_score_rows(z, 5000, sd.DTYPES["bf16"], 20, 5000, 0.9, token, logp, None, None, stream=side.cuda_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd.sd_score_rows(z, 5000, sd.DTYPES["bf16"], 20, 5000, 0.9, token, None, rank, None,
                         stream=torch.cuda.current_stream().cuda_stream)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((logp, rank, H, ids, lps), want):
        assert np.array_equal(a.cpu().numpy(), b)


# ------------------------------------------------------------------ as they are used

def test_rollouts_of_a_prompt(sd, ws):
    """A prompt's pages forked into rollouts, tokens written and attended, the worst rollouts ended and the best forked, the
    pool compacted: at every step each rollout attends to its own history, kept apart in 64 bits."""
    g, rng = gen(20), np.random.default_rng(20)
    H, Hkv, hd, ps, n_pages, V = 8, 4, 128, 16, 600, 900
    kc, vc = (torch.full((n_pages, Hkv, ps, hd), float("nan"), device="cuda", dtype=torch.float16) for _ in range(2))
    cache, width = sd.Pages.of(kc, vc), 90
    new = lambda *s: torch.full(s, -1, dtype=torch.int32, device="cuda")
    n0 = 1100
    table, lens, free = new(1, width), i32([0]), i32(rng.permutation(n_pages))
    history = [(torch.zeros(0, Hkv, hd, device="cuda", dtype=torch.float16),) * 2]
    scale = 1 / math.sqrt(hd)
    score = torch.zeros(1, device="cuda")
    for step in range(12):
        # ---- fork: the prompt into six, later the best two into two each and the worst ended
        R = lens.numel()
        if step == 1:
            parent = [0] * 6
        elif step > 1:
            order = torch.argsort(score, descending=True, stable=True).tolist()
            parent = [order[0], order[1], order[0], order[2], order[1], order[3]]
        else:
            parent = [0]
        N = len(parent)
        t2, l2, copies, ref, f2, info = new(N, width), new(N), new(N, 3), new(n_pages), new(n_pages), new(4)
        sd.sd_page_fork(table, width, lens, R, i32(parent), N, free, free.numel(), ps, n_pages, t2, l2, copies, ref, f2, info,
                        new(sd.sd_page_work(R, N, n_pages)))
        sd.sd_page_copy([cache], copies, info, N)
        history, score = [history[p] for p in parent], score[torch.tensor(parent, device="cuda")]
        table, lens = t2, l2
        free = f2[:info[1].item()].contiguous()
        assert info[2].item() == 0
        if step == 7:
            t3, ref3, f3 = new(N, width), new(n_pages), new(n_pages)
            moves = new(n_pages // 2, 3)
            sd.sd_page_compact(table, width, lens, N, ps, n_pages, t3, moves, ref3, f3, info, new(sd.sd_page_work(N, 0, n_pages)))
            sd.sd_page_copy([cache], moves, info, moves.shape[0])
            table, free = t3, f3[:info[1].item()].contiguous()
            assert table.max().item() == info[3].item() - 1 and info[3].item() + free.numel() == n_pages
        # ---- new tokens
        count = n0 if step == 0 else 1
        rows = N * count
        total, start, slot, pos, req, pinfo = new(N), new(N + 1), new(rows), new(rows), new(rows), new(4)
        sd.sd_page_plan(lens, i32([count] * N), N, free, free.numel(), ps, table, width, rows, total, start, slot, pos, req, pinfo)
        free = free[pinfo[1].item():].contiguous()
        k, v = randn(g, rows, Hkv, hd, dt="f16"), randn(g, rows, Hkv, hd, dt="f16")
        sd.sd_rope_write_pages(None, None, 0, slot, rows, sd.DTYPES["f16"], None, 0, None, 0, 0, k, v, Hkv * hd, cache)
        lens = total
        history = [(torch.cat([a, k[i * count:(i + 1) * count]]), torch.cat([b, v[i * count:(i + 1) * count]]))
                   for i, (a, b) in enumerate(history)]
        # ---- attention over the prompt's full pages once, and over the own ones
        q = randn(g, N, H, hd, dt="f16")
        out, lse = run_shared(sd, ws, q, cache, table, lens, i32([0, N]), i32([n0 // ps if step else 0]), scale)
        check_rows(q, history, out, lse, Hkv, scale, "f16", "f16")
        # ---- scores
        z = out.float().reshape(N, H * hd) @ torch.randn(H * hd, V, generator=g, device="cuda")
        token = i32(rng.integers(0, V, N))
        logp = torch.empty(N, device="cuda")
        sd.sd_score_rows(z, V, sd.DTYPES["f32"], N, V, 1.0, token, logp, None, None)
        want = torch.log_softmax(z.double(), -1)[torch.arange(N, device="cuda"), token.long()]
        assert all(near(a, b) for a, b in zip(logp.tolist(), want.tolist()))
        score = score + logp
