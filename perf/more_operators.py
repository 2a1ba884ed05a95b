"""Workloads of rollouts over the paged cache: pages forked, compacted and copied,
attention that reads a common prefix once, and scores of tokens.

Five operators, each in its plain form (elementary torch operations in 32 bits)
and through the library's entry points:

* ``fork``    -- rows of the next step from rows of this one: tables, lengths, copies,
  reference counts and the free list (``sd_page_fork``);
* ``compact`` -- the pages in use moved to the front of the pool (``sd_page_compact``);
* ``copy``    -- pages copied in every layer's cache (``sd_page_copy``);
* ``shared``  -- attention of one new token per request where groups of requests
  share their first pages (``sd_attend_shared``);
* ``score``   -- log probability and rank of given tokens, entropy, and the most
  probable alternatives (``sd_score_rows``).

Lengths, groups and parents are fixed lists of the case; page ids and values are
drawn from the seed, so that the work of a case is the same for every seed.
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a 300-token prompt forked into 16 rollouts
        dict(name="fork_g16", op="fork", requests=1, beams=1, fan=16, low=300, high=300, common=0, ended=0, page=16,
             spare=7),
        # beam search of 500 requests with 4 beams each: parents drawn within a request, 40 requests end
        dict(name="fork_beams_2000", op="fork", requests=500, beams=4, fan=1, low=1, high=3000, common=60, ended=40,
             page=16, spare=5000),
        # the pool of 16 rollouts after other requests have left it
        dict(name="compact_g16", op="compact", R=16, low=301, high=425, page=16, pool=1024),
        # a server's pool at a third of its pages
        dict(name="compact_2000", op="compact", R=2000, low=0, high=8000, page=64, pool=150011),
        # the partly filled last page of a 300-token prompt for 15 more rollouts, 28 layers, 8 kv heads of 128
        dict(name="copy_fork_28_layers", op="copy", copies=15, layers=28, Hkv=8, hd=128, cache="f16", page=16,
             positions=12, pool=64),
        # whole pages moved by a compaction, one layer
        dict(name="copy_compact_2000", op="copy", copies=2000, layers=1, Hkv=8, hd=128, cache="bf16", page=64,
             positions=64, pool=4103),
        # 16 rollouts of a 300-token prompt, up to 125 own positions, 16 query / 8 kv heads of 128
        dict(name="shared_g16_425", op="shared", groups=1, small=16, large=16, near=300, far=300, own_low=1,
             own_high=125, loose=0, H=16, Hkv=8, hd=128, dt="f16", cache="f16", page=16),
        # 64 rollouts of a longer prompt on the GPT-2-Medium shape: fp32 activations, fp16 cache
        dict(name="shared_g64_2000", op="shared", groups=1, small=64, large=64, near=2000, far=2000, own_low=0,
             own_high=250, loose=0, H=16, Hkv=16, hd=64, dt="f32", cache="f16", page=32),
        # groups of 2 to 32 requests behind prefixes of 1000 to 16000 positions, 8 query heads to a kv head, and three
        # requests of their own
        dict(name="shared_groups_16k", op="shared", groups=8, small=2, large=32, near=1000, far=16000, own_low=1,
             own_high=500, loose=3, H=64, Hkv=8, hd=128, dt="bf16", cache="bf16", page=64),
        # one frame's codes of 16 rollouts: the code predictor's vocabulary
        dict(name="score_g16_2048", op="score", rows=16, V=2048, dt="f32", top=5, T=0.9, masked=0.0, pad=0, peaked=0.3),
        # the speech tokens of two 400-step runs, scored with alternatives
        dict(name="score_800_8194", op="score", rows=800, V=8194, dt="f32", top=20, T=0.8, masked=0.0, pad=13,
             peaked=0.3),
        # a padded batch over a large text vocabulary, a fifth of it masked
        dict(name="score_1021_of_128k", op="score", rows=1021, V=131075, dt="bf16", top=8, T=1.0, masked=0.2, pad=100,
             peaked=0.5),
    ]


def _log(rng, a, b):
    """A whole number between a and b, spread over the logarithm."""
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


HEADS = [(16, 16, 64), (16, 8, 128), (16, 4, 64), (32, 8, 128), (12, 12, 64), (16, 1, 128), (40, 8, 128), (64, 8, 128)]


def draw(rng):
    op = rng.choice(["fork", "compact", "copy", "shared", "score"])
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "fork":
        requests = _log(rng, 1, 500)
        high = _log(rng, 1, 4000)
        return dict(op=op, requests=requests, beams=rng.choice([1, 2, 3, 4]), fan=rng.choice([1, 1, 2, 4]),
                    low=rng.randint(1, high), high=high, common=rng.randint(0, 100), ended=rng.randint(0, requests // 4),
                    page=page, spare=rng.randint(0, 3000))
    if op == "compact":
        R = _log(rng, 1, 2000)
        return dict(op=op, R=R, low=0, high=_log(rng, 4, 8000), page=page, pool=_log(rng, 64, 150000))
    if op == "copy":
        copies = _log(rng, 1, 1000)
        H, Hkv, hd = rng.choice(HEADS)
        return dict(op=op, copies=copies, layers=_log(rng, 1, max(1, min(30, 2000 // copies))), Hkv=Hkv, hd=hd,
                    cache=rng.choice(["f16", "bf16", "e4m3"]), page=page, positions=rng.randint(1, page),
                    pool=2 * copies + rng.randint(0, 50))
    if op == "shared":
        H, Hkv, hd = rng.choice(HEADS)
        dt, cache = rng.choice([("f32", "f16"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3")])
        groups = _log(rng, 1, 8)
        large = _log(rng, 1, 96 // groups)
        far = _log(rng, 16, 8000)
        return dict(op=op, groups=groups, small=rng.randint(1, large), large=large, near=rng.randint(1, far), far=far,
                    own_low=rng.randint(0, 20), own_high=rng.randint(20, 500), loose=rng.randint(0, 4), H=H, Hkv=Hkv,
                    hd=hd, dt=dt, cache=cache, page=page)
    V = _log(rng, 200, 200000)
    return dict(op=op, rows=_log(rng, 1, max(1, min(4000, 100000000 // V))), V=V, dt=rng.choice(["f32", "f16", "bf16"]),
                top=rng.randint(1, 32), T=rng.choice([0.8, 0.9, 1.0]), masked=rng.choice([0.0, 0.2, 0.7]),
                pad=rng.randint(0, 3), peaked=rng.choice([0.0, 0.3, 0.6]))


def _spread(n, low, high):
    """n numbers from low to high, evenly spread over the logarithm where that spans more than a factor of ten."""
    if n <= 0:
        return []
    if n == 1:
        return [high]
    a = max(low, 1)
    if high > 10 * a:
        v = [int(round(a * (high / a) ** (i / (n - 1)))) for i in range(n)]
    else:
        v = [int(round(low + (high - low) * i / (n - 1))) for i in range(n)]
    if low == 0:
        v[0] = 0
    return v


def _pages(n, page):
    return -(-n // page)


def _fork_rows(case):
    """(length of every row, pages in common of every request, parent of every new row)."""
    n, beams = case["requests"], case["beams"]
    each = _spread(n, case["low"], case["high"])
    step = next(s for s in range(n // 2 + 1, 2 * n + 2) if math.gcd(s, n) == 1)
    each = [each[(i * step) % n] for i in range(n)]
    common = [min(case["common"], x // case["page"]) for x in each]
    length = [x for x in each for _ in range(beams)]
    rng = random.Random(n * 131 + beams)
    ended = set(rng.sample(range(n), case["ended"]))
    parent = []
    for r in range(n):
        for _ in range(beams * case["fan"]):
            parent.append(-1 if r in ended else r * beams + rng.randrange(beams))
    return length, common, parent


def _fork_sizes(case):
    """(pages in use, copies, width of a table row)."""
    length, common, parent = _fork_rows(case)
    pg, beams = case["page"], case["beams"]
    used = sum(common) + sum(_pages(x, pg) - common[r // beams] for r, x in enumerate(length))
    seen, copies = set(), 0
    for p in parent:
        if p >= 0 and length[p] % pg:
            copies += p in seen
            seen.add(p)
    return used, copies, max(_pages(x, pg) for x in length) + 3


def _compact_lengths(case):
    """Lengths whose pages the pool holds."""
    v = _spread(case["R"], case["low"], case["high"])
    most = case["pool"] * 2 // 3
    while sum(_pages(x, case["page"]) for x in v) > most:
        v = [x // 2 for x in v]
    return v


def _groups(case):
    """(size of every group, its prefix, length of every request, pages in common of every group)."""
    size = _spread(case["groups"], case["small"], case["large"])
    prefix = _spread(case["groups"], case["near"], case["far"])[::-1]
    R = sum(size) + case["loose"]
    mine = _spread(R, case["own_low"], case["own_high"])
    step = next(s for s in range(R // 2 + 1, 2 * R + 2) if math.gcd(s, R) == 1)
    mine = [mine[(i * step) % R] for i in range(R)]
    length, at = [], 0
    for n, p in zip(size, prefix):
        length += [p + x for x in mine[at:at + n]]
        at += n
    return size, prefix, length + mine[at:], [p // case["page"] for p in prefix]


def work(case):
    op = case["op"]
    if op == "fork":
        length, common, parent = _fork_rows(case)
        used, copies, width = _fork_sizes(case)
        pool, N = used + copies + case["spare"], len(parent)
        old = sum(_pages(x, case["page"]) for x in length)
        # used entries, lengths, parents and the free list in; rows, lengths, counts, copies and the free list out
        return {"bytes": 4 * (old + len(length) + N + pool - used) + 4 * (N * width + N + pool + 3 * copies) +
                4 * (pool - used), "flops": 2 * N * width}
    if op == "compact":
        L = _compact_lengths(case)
        held = sum(_pages(x, case["page"]) for x in L)
        width = max(1, max(_pages(x, case["page"]) for x in L)) + 3
        return {"bytes": 4 * (held + len(L)) + 4 * (len(L) * width + 2 * case["pool"] - held), "flops": 2 * held}
    if op == "copy":
        n = case["copies"] * case["layers"] * case["Hkv"] * case["positions"] * case["hd"] * 2
        return {"bytes": 2 * n * SIZE[case["cache"]] + 12 * case["copies"], "flops": 0}
    if op == "shared":
        size, prefix, length, common = _groups(case)
        pg, hd = case["page"], case["hd"]
        once = sum(c * pg for c in common)
        alone = sum(length) - sum(n * c * pg for n, c in zip(size, common))
        R = len(length)
        return {"bytes": 2 * (once + alone) * case["Hkv"] * hd * SIZE[case["cache"]] +
                2 * R * case["H"] * hd * SIZE[case["dt"]] + 4 * (once + alone) // pg,
                "flops": 4 * sum(length) * case["H"] * hd}
    n = case["rows"] * case["V"]
    return {"bytes": n * SIZE[case["dt"]] + case["rows"] * (16 + 8 * case["top"]), "flops": 6 * n}


# ------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _blank(*shape):
    return torch.full(shape, -1, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)

    def normal(*shape, dt="f32", scale=1.0):
        x = torch.empty(*shape, dtype=torch.float16 if dt == "e4m3" else DT[dt], device="cuda")
        x.normal_(0.0, scale, generator=g)
        return x.to(DT[dt])

    op = case["op"]
    st = dict(case=case, op=op)
    if op == "fork":
        length, common, parent = _fork_rows(case)
        used, copies, width = _fork_sizes(case)
        pg, beams, R, N = case["page"], case["beams"], len(length), len(parent)
        pool = used + copies + case["spare"]
        ids = torch.randperm(pool, generator=h).to(torch.int32).numpy()
        table = np.full((R, width), -1, np.int32)
        at = 0
        for r in range(R):
            c, n = common[r // beams], _pages(length[r], pg)
            if r % beams == 0:
                shared = ids[at:at + c]
                at += c
            table[r, :c] = shared
            table[r, c:n] = ids[at:at + n - c]
            at += n - c
        st.update(table=torch.from_numpy(table).cuda(), len=_ints(length), parent=_ints(parent), page=pg, pool=pool,
                  free=torch.from_numpy(ids[at:].copy()).cuda(), table_out=_blank(N, width), len_out=_blank(N),
                  copies=_blank(N, 3), ref=_blank(pool), free_out=_blank(pool), info=_blank(4))
        if own:
            import autoregressive_speech_token_gb300 as sd
            st["work"] = _blank(sd.sd_page_work(R, N, pool))
    elif op == "compact":
        L, pg, pool = _compact_lengths(case), case["page"], case["pool"]
        order = torch.randperm(len(L), generator=h).tolist()
        L = [L[i] for i in order]
        width = max(1, max(_pages(x, pg) for x in L)) + 3
        held = sum(_pages(x, pg) for x in L)
        table = torch.full((len(L), width), -1, dtype=torch.int32)
        owned = torch.arange(width)[None, :] < torch.tensor([_pages(x, pg) for x in L])[:, None]
        table[owned] = torch.randperm(pool, generator=h)[:held].to(torch.int32)
        st.update(table=table.cuda(), len=_ints(L), page=pg, pool=pool, table_out=_blank(len(L), width),
                  copies=_blank(pool // 2 + 1, 3), ref=_blank(pool), free_out=_blank(pool), info=_blank(4))
        if own:
            import autoregressive_speech_token_gb300 as sd
            st["work"] = _blank(sd.sd_page_work(len(L), 0, pool))
    elif op == "copy":
        n, pg = case["copies"], case["page"]
        ids = torch.randperm(case["pool"], generator=h)[:2 * n].to(torch.int32)
        pairs = torch.stack([ids[:n], ids[n:], torch.full((n,), case["positions"], dtype=torch.int32)], 1)
        shape = (case["pool"], case["Hkv"], pg, case["hd"])
        st.update(pairs=pairs.contiguous().cuda(), count=_ints([n]), page=pg,
                  k=[normal(*shape, dt=case["cache"]) for _ in range(case["layers"])],
                  v=[normal(*shape, dt=case["cache"]) for _ in range(case["layers"])])
        if own:
            import autoregressive_speech_token_gb300 as sd
            st["caches"] = sd.PageArray.of([sd.Pages.of(k, v) for k, v in zip(st["k"], st["v"])])
    elif op == "shared":
        H, Hkv, hd, pg = case["H"], case["Hkv"], case["hd"], case["page"]
        size, prefix, length, common = _groups(case)
        R = len(length)
        shared = [c for n, c in zip(size, common) for _ in range(n)] + [0] * case["loose"]
        held = sum(common) + sum(_pages(x, pg) - c for x, c in zip(length, shared))
        ids = torch.randperm(held + 11, generator=h).to(torch.int32)
        width = max(1, max(_pages(x, pg) for x in length)) + 1
        table = torch.full((R, width), -1, dtype=torch.int32)
        at = r = 0
        for n, c in zip(size + [1] * case["loose"], common + [0] * case["loose"]):
            first = ids[at:at + c]
            at += c
            for _ in range(n):
                k = _pages(length[r], pg)
                table[r, :c] = first
                table[r, c:k] = ids[at:at + k - c]
                at += k - c
                r += 1
        starts = [sum(size[:i]) for i in range(len(size) + 1)]
        st.update(q=normal(R, H, hd, dt=case["dt"]), kc=normal(held + 11, Hkv, pg, hd, dt=case["cache"]),
                  vc=normal(held + 11, Hkv, pg, hd, dt=case["cache"]), table=table.cuda(), len=_ints(length),
                  group=_ints(starts), common=_ints(common), scale=1.0 / math.sqrt(hd),
                  out=torch.empty(R, H, hd, dtype=DT[case["dt"]], device="cuda"), ks=None, vs=None)
        if case["cache"] == "e4m3":
            st["ks"] = torch.rand(Hkv, generator=g, device="cuda") * 0.5 + 0.75
            st["vs"] = torch.rand(Hkv, generator=g, device="cuda") * 0.5 + 0.75
        if own:
            import autoregressive_speech_token_gb300 as sd
            st["cache"] = sd.Pages.of(st["kc"], st["vc"], st["ks"], st["vs"])
            st["ws"] = sd.AttnWorkspace()
            st["dtype"] = sd.DTYPES[case["dt"]]
    else:
        rows, V, top = case["rows"], case["V"], case["top"]
        z = normal(rows, V, dt="f32", scale=2.5)
        token = torch.randint(0, V, (rows,), generator=g, device="cuda")
        sharp = torch.rand(rows, generator=g, device="cuda") < case["peaked"]
        z[torch.arange(rows, device="cuda"), token] += torch.where(sharp, 12.0, 0.0)
        if case["masked"]:
            # the same part of the vocabulary in every row, but for the row's own token
            keep = z.gather(1, token[:, None])
            z.masked_fill_(torch.rand(V, generator=g, device="cuda")[None, :] < case["masked"], float("-inf"))
            z.scatter_(1, token[:, None], keep)
        token[rows - min(case["pad"], rows - 1):] = -1
        f = dict(dtype=torch.float32, device="cuda")
        st.update(z=z.to(DT[case["dt"]]), token=token.to(torch.int32), top=top, T=case["T"],
                  logp=torch.empty(rows, **f), rank=_blank(rows), entropy=torch.empty(rows, **f),
                  top_id=_blank(rows, top), top_logp=torch.empty(rows, top, **f))
        if own:
            import autoregressive_speech_token_gb300 as sd
            st["dtype"] = sd.DTYPES[case["dt"]]
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _own[st["op"]](st) if own else _plain[st["op"]](st)


def _behind(buffer, x):
    """`buffer` (blank) with x at its front."""
    out = torch.full_like(buffer, -1)
    out[:x.shape[0]] = x.to(torch.int32)
    return out


def _plain_fork(st):
    table, ln, parent, pg, free = st["table"], st["len"].long(), st["parent"].long(), st["page"], st["free"]
    R, width = table.shape
    N = parent.numel()
    dev = table.device
    live = (parent >= 0) & (parent < R)
    p = parent.clamp(0, R - 1)
    n = torch.where(live, ln[p], torch.zeros_like(p))
    full, rest = n // pg, n % pg
    col = torch.arange(width, device=dev)[None, :]
    out = torch.where(col < ((n + pg - 1) // pg)[:, None], table[p], torch.full_like(table[p], -1))
    i = torch.arange(N, device=dev)
    first = torch.full((R,), N, dtype=torch.int64, device=dev).scatter_reduce(
        0, p, torch.where(live, i, torch.full_like(i, N)), "amin")
    need = live & (rest > 0) & (first[p] != i)
    rows = torch.nonzero(need)[:, 0]
    taken = rows.numel()
    source = out[rows, full[rows]]
    out[rows, full[rows]] = free[:taken]
    copies = torch.stack([source.long(), free[:taken].long(), rest[rows]], 1)
    ref = torch.zeros(st["pool"], dtype=torch.int64, device=dev)
    named = out[out >= 0].long()
    ref.index_add_(0, named, torch.ones_like(named))
    before = torch.zeros(st["pool"], dtype=torch.bool, device=dev)
    before[table[col < ((ln + pg - 1) // pg)[:, None]].long()] = True
    back = torch.nonzero(before & (ref == 0))[:, 0]
    free_out = torch.cat([free[taken:].long(), back])
    info = torch.tensor([taken, free_out.numel(), 0, 0], dtype=torch.int32, device=dev)
    info[3] = n.max()
    return [out, n.to(torch.int32), _behind(st["copies"], copies), ref.to(torch.int32),
            _behind(st["free_out"], free_out), info]


def _plain_compact(st):
    table, ln, pg, pool = st["table"], st["len"].long(), st["page"], st["pool"]
    dev = table.device
    used = torch.arange(table.shape[1], device=dev)[None, :] < ((ln + pg - 1) // pg)[:, None]
    ref = torch.zeros(pool, dtype=torch.int64, device=dev)
    named = table[used].long()
    ref.index_add_(0, named, torch.ones_like(named))
    live = ref > 0
    n = live.sum()
    ids = torch.arange(pool, device=dev)
    source = torch.nonzero(live & (ids >= n))[:, 0]
    target = torch.nonzero(~live & (ids < n))[:, 0]
    to = ids.clone()
    to[source] = target
    out = torch.where(used, to[table.clamp(min=0).long()], torch.full_like(to[:1], -1)).to(torch.int32)
    moved = torch.zeros_like(ref)
    moved[to[live]] = ref[live]
    copies = torch.stack([source, target, torch.full_like(source, pg)], 1)
    info = torch.stack([torch.full_like(n, source.numel()), pool - n, torch.zeros_like(n), n]).to(torch.int32)
    return [out, _behind(st["copies"], copies), moved.to(torch.int32), _behind(st["free_out"], ids[n:]), info]


def _plain_copy(st):
    pairs = st["pairs"].long()
    live = torch.arange(st["page"], device=pairs.device)[None, :] < pairs[:, 2:]
    for pool in st["k"] + st["v"]:
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        raw[pairs[:, 1]] = torch.where(live[:, None, :, None], raw[pairs[:, 0]], raw[pairs[:, 1]])
    return st["k"], st["v"]


def _plain_shared(st):
    c, table = st["case"], st["table"].long().clamp(min=0)
    H, Hkv, hd = c["H"], c["Hkv"], c["hd"]
    R = table.shape[0]

    def gather(pool, scale):
        if pool.dtype == torch.float8_e4m3fn:
            x = pool.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        else:
            x = pool[table].float()
        x = x.permute(0, 2, 1, 3, 4).reshape(R, Hkv, -1, hd)
        return x if scale is None else x * scale[None, :, None, None]

    k, v = gather(st["kc"], st["ks"]), gather(st["vc"], st["vs"])
    live = torch.arange(k.shape[2], device="cuda")[None, :] < st["len"][:, None]
    v = v.masked_fill_(~live[:, None, :, None], 0.0)
    s = torch.matmul(st["q"].float().reshape(R, Hkv, H // Hkv, hd), k.transpose(-1, -2)) * st["scale"]
    s = s.masked_fill_(~live[:, None, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(den == 0, torch.ones_like(den), den)
    st["out"].copy_(o.reshape(R, H, hd))
    return st["out"]


def _plain_score(st):
    z, top = st["z"].float(), st["top"]
    rows, V = z.shape
    x = z / st["T"]
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(1, keepdim=True)
    lse = m + torch.log(s)
    entropy = torch.log(s[:, 0]) - (torch.where(e > 0, x - m, torch.zeros_like(x)) * e).sum(1) / s[:, 0]
    t = st["token"].long()
    given = t >= 0
    zt = z.gather(1, t.clamp(min=0)[:, None])
    logp = torch.where(given, (zt / st["T"] - lse)[:, 0], torch.zeros_like(entropy))
    ahead = (z > zt) | ((z == zt) & (torch.arange(V, device=z.device)[None, :] < t[:, None]))
    rank = torch.where(given, ahead.sum(1), -1).to(torch.int32)
    value, index = torch.sort(z, dim=1, descending=True, stable=True)
    value, index = value[:, :top], index[:, :top]
    if value.shape[1] < top:
        more = (0, top - value.shape[1])
        value = torch.nn.functional.pad(value, more, value=float("-inf"))
        index = torch.nn.functional.pad(index, more, value=-1)
    index = torch.where(value == float("-inf"), -1, index).to(torch.int32)
    return logp, rank, entropy, index, value / st["T"] - lse


_plain = dict(fork=_plain_fork, compact=_plain_compact, copy=_plain_copy, shared=_plain_shared, score=_plain_score)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _own_fork(st):
    import autoregressive_speech_token_gb300 as sd
    R, width = st["table"].shape
    sd.sd_page_fork(st["table"], width, st["len"], R, st["parent"], st["parent"].numel(), st["free"],
                    st["free"].numel(), st["page"], st["pool"], st["table_out"], st["len_out"], st["copies"],
                    st["ref"], st["free_out"], st["info"], st["work"], _stream())
    return [st[x] for x in ("table_out", "len_out", "copies", "ref", "free_out", "info")]


def _own_compact(st):
    import autoregressive_speech_token_gb300 as sd
    R, width = st["table"].shape
    sd.sd_page_compact(st["table"], width, st["len"], R, st["page"], st["pool"], st["table_out"], st["copies"],
                       st["ref"], st["free_out"], st["info"], st["work"], _stream())
    return [st[x] for x in ("table_out", "copies", "ref", "free_out", "info")]


def _own_copy(st):
    import autoregressive_speech_token_gb300 as sd
    sd.sd_page_copy(st["caches"], st["pairs"], st["count"], st["pairs"].shape[0], _stream())
    return st["k"], st["v"]


def _own_shared(st):
    import autoregressive_speech_token_gb300 as sd
    R, H, hd = st["q"].shape
    sd.sd_attend_shared(st["ws"], st["cache"], st["table"], st["table"].shape[1], st["len"], R, st["group"],
                        st["common"], st["common"].numel(), st["dtype"], st["q"], H * hd, H, st["scale"], st["out"],
                        H * hd, None, _stream())
    return st["out"]


def _own_score(st):
    import autoregressive_speech_token_gb300 as sd
    rows, V = st["z"].shape
    sd.sd_score_rows(st["z"], V, st["dtype"], rows, V, st["T"], st["token"], st["logp"], st["rank"], st["entropy"],
                     st["top"], st["top_id"], st["top_logp"], _stream())
    return [st[x] for x in ("logp", "rank", "entropy", "top_id", "top_logp")]


_own = dict(fork=_own_fork, compact=_own_compact, copy=_own_copy, shared=_own_shared, score=_own_score)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))


def _front(buffer, rows):
    out = np.full(tuple(buffer.shape), -1, np.int64)
    if len(rows):
        out[:len(rows)] = rows
    return out


def _out(*xs):
    return [torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in xs]


def _exact_fork(st):
    table, ln, parent, free = (st[x].cpu().numpy().astype(np.int64) for x in ("table", "len", "parent", "free"))
    pg, pool = st["page"], st["pool"]
    out = np.full((len(parent), table.shape[1]), -1, np.int64)
    length, copies, seen = np.zeros(len(parent), np.int64), [], set()
    for i, p in enumerate(parent):
        if not 0 <= p < len(ln):
            continue
        n = length[i] = ln[p]
        k = -(-n // pg)
        out[i, :k] = table[p, :k]
        if n % pg:
            if p in seen:
                page = free[len(copies)]
                copies.append((out[i, k - 1], page, n % pg))
                out[i, k - 1] = page
            seen.add(p)
    ref = np.bincount(out[out >= 0], minlength=pool)
    old = set()
    for r, n in enumerate(ln):
        old.update(table[r, :-(-n // pg)].tolist())
    left = free[len(copies):].tolist() + sorted(x for x in old if ref[x] == 0)
    return _out(out, length, _front(st["copies"], copies), ref, _front(st["free_out"], left),
                [len(copies), len(left), 0, length.max()])


def _exact_compact(st):
    table, ln = st["table"].cpu().numpy().astype(np.int64), st["len"].cpu().numpy().astype(np.int64)
    pg, pool = st["page"], st["pool"]
    count = np.zeros(pool, np.int64)
    for r, n in enumerate(ln):
        for x in table[r, :-(-n // pg)]:
            count[x] += 1
    live = [x for x in range(pool) if count[x]]
    n = len(live)
    moves = dict(zip([x for x in live if x >= n], [x for x in range(n) if not count[x]]))
    out = np.full(table.shape, -1, np.int64)
    ref = np.zeros(pool, np.int64)
    for r, m in enumerate(ln):
        for j in range(-(-m // pg)):
            out[r, j] = moves.get(table[r, j], table[r, j])
            ref[out[r, j]] += 1
    copies = [(a, b, pg) for a, b in moves.items()]
    return _out(out, _front(st["copies"], copies), ref, _front(st["free_out"], range(n, pool)),
                [len(copies), pool - n, 0, n])


def _exact_copy(st):
    for pool in st["k"] + st["v"]:
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        for a, b, n in st["pairs"].tolist():
            raw[b, :, :n] = raw[a, :, :n]
    return st["k"], st["v"]


def _exact_shared(st):
    c = st["case"]
    H, Hkv, hd, pg = c["H"], c["Hkv"], c["hd"], c["page"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for r, n in enumerate(st["len"].tolist()):
        if n == 0:
            continue
        ids = st["table"][r, :_pages(n, pg)].tolist()

        def rows(pool, scale):
            x = torch.cat([pool[i].double().transpose(0, 1) for i in ids])[:n]
            return x if scale is None else x * scale.double()[None, :, None]

        q = st["q"][r].double().reshape(Hkv, H // Hkv, hd)
        s = torch.einsum("gmd,lgd->gml", q, rows(st["kc"], st["ks"])) * st["scale"]
        out[r] = torch.einsum("gml,lgd->gmd", torch.softmax(s, -1), rows(st["vc"], st["vs"])).reshape(H, hd)
    return out


def _exact_score(st):
    rows, V = st["z"].shape
    top = st["top"]
    logp = torch.zeros(rows, dtype=torch.float64, device="cuda")
    entropy = torch.zeros_like(logp)
    rank, index = [], np.full((rows, top), -1, np.int64)
    value = torch.full((rows, top), float("-inf"), dtype=torch.float64, device="cuda")
    token = st["token"].tolist()
    for r in range(rows):
        z = st["z"][r].double()
        logs = torch.log_softmax(z / float(np.float32(st["T"])), 0)
        p = torch.exp(logs)
        entropy[r] = -(p * torch.where(p > 0, logs, torch.zeros_like(logs))).sum()
        t = token[r]
        rank.append(-1)
        if t >= 0:
            logp[r] = logs[t]
            rank[-1] = int((z > z[t]).sum() + (z[:t] == z[t]).sum())
        # what can be among the first: at or above the value in place `top`, in order of the index
        if top:
            bound = torch.topk(z, min(top, V)).values[-1]
            some = torch.nonzero((z >= bound) & (z > float("-inf")))[:, 0].cpu().numpy()
            zs = z.cpu().numpy()[some]
            best = some[np.lexsort((some, -zs))][:top]
            index[r, :len(best)] = best
            value[r, :len(best)] = logs[torch.from_numpy(best).cuda()]
    return [logp] + _out(rank) + [entropy] + _out(index) + [value]


_exact = dict(fork=_exact_fork, compact=_exact_compact, copy=_exact_copy, shared=_exact_shared, score=_exact_score)
