"""Workloads of the paged key-value cache and of cross attention.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and through the library's entry points:

* ``plan``  -- block tables, slot maps and positions of a step, from the
  requests' lengths (``sd_page_plan``);
* ``write`` -- rotary positions (one or several axes) of q and k, and the write
  of k and v into the cache's pages (``sd_rope_write_pages``);
* ``pages`` -- attention of one new token per request over the paged cache
  (``sd_attend_pages``);
* ``cross`` -- attention of [B][Lq] queries to an encoder's states [B][Lk] with
  a length per batch row (``sd_attend_cross``).

A request's lengths are a fixed list of the case in an order drawn from the
seed, so that the work of a case is the same for every seed.
"""

import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the step of 16 rollouts of one prompt (300 prompt tokens, up to 125 frames), one new token each
        dict(name="plan_step_g16", op="plan", R=16, low=300, high=425, prompts=0, longest=0, idle=0, page=16),
        # a busy server's step: 2000 requests, most with one new token, 200 with a prompt, 100 that wait
        dict(name="plan_mixed_2000", op="plan", R=2000, low=0, high=8000, prompts=200, longest=2048, idle=100,
             page=64),
        # the same 16 rollouts' q, k, v of one layer (16 query / 8 kv heads of 128, fp32 activations, fp16 cache)
        dict(name="write_step_g16", op="write", n=16, skipped=0, H=16, Hkv=8, hd=128, dt="f32", cache="f16", page=16,
             axes=1, interleaved=False, theta=1e4, far=512),
        # long prompts with time, height and width positions, taken out of a fused q|k|v projection's rows
        dict(name="write_prompt_axes3", op="write", n=30011, skipped=523, H=16, Hkv=8, hd=128, dt="bf16",
             cache="bf16", page=64, axes=3, interleaved=True, theta=1e6, far=32768),
        # one stream of the GPT-2-Medium-shaped decoder near its 400th position
        dict(name="pages_one_399", op="pages", R=1, low=399, high=399, empty=0, H=16, Hkv=16, hd=64, dt="f32",
             cache="f16", page=16),
        # 16 rollouts of the Talker shape
        dict(name="pages_g16_425", op="pages", R=16, low=301, high=425, empty=0, H=16, Hkv=8, hd=128, dt="f16",
             cache="f16", page=16),
        # requests of every length up to 32768, two of them without any position yet
        dict(name="pages_ragged_32k", op="pages", R=48, low=1, high=32768, empty=2, H=16, Hkv=8, hd=128, dt="bf16",
             cache="bf16", page=64),
        # a full batch on an 8-bit cache with 8 query heads to a kv head
        dict(name="pages_e4m3_4100", op="pages", R=64, low=2000, high=4100, empty=0, H=64, Hkv=8, hd=128, dt="bf16",
             cache="e4m3", page=32),
        # the single-token step of a decoder that attends to its encoder's states, a padded batch of 16
        dict(name="cross_step_b16", op="cross", B=16, Lq=1, Lk=1500, low=0, H=16, Hkv=16, hd=64, dt="f16", kv="f16"),
        # 32 learned queries over 150 conditioning states (fp32 activations)
        dict(name="cross_32_over_150", op="cross", B=2, Lq=32, Lk=150, low=97, H=16, Hkv=16, hd=64, dt="f32",
             kv="f16"),
        # a padded batch of prompts over encoder states of other lengths, odd sizes
        dict(name="cross_777_over_1500", op="cross", B=8, Lq=777, Lk=1500, low=211, H=16, Hkv=16, hd=64, dt="bf16",
             kv="bf16"),
        # long inputs, grouped heads of 128
        dict(name="cross_8192_over_8190", op="cross", B=2, Lq=8192, Lk=8190, low=8000, H=16, Hkv=8, hd=128, dt="bf16",
             kv="bf16"),
    ]


def _log(rng, a, b):
    """A whole number between a and b, spread over the logarithm."""
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


HEADS = [(16, 16, 64), (16, 8, 128), (16, 4, 64), (32, 8, 128), (12, 12, 64), (16, 1, 128), (40, 8, 128), (64, 4, 64)]


def draw(rng):
    op = rng.choice(["plan", "write", "pages", "cross"])
    if op == "plan":
        R = _log(rng, 1, 2000)
        return dict(op=op, R=R, low=0, high=_log(rng, 16, 8000), prompts=rng.randint(0, R // 10),
                    longest=_log(rng, 2, 2048), idle=rng.randint(0, R // 4), page=rng.choice([8, 16, 32, 64, 128]))
    H, Hkv, hd = rng.choice(HEADS)
    if op == "write":
        n = _log(rng, 1, 8000)
        dt, cache = rng.choice([("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")])
        return dict(op=op, n=n, skipped=rng.randint(0, n // 4), H=H, Hkv=Hkv, hd=hd, dt=dt, cache=cache,
                    page=rng.choice([8, 16, 32, 64, 128]), axes=rng.choice([1, 2, 3, 4]),
                    interleaved=rng.random() < 0.5, theta=rng.choice([1e4, 1e6]), far=_log(rng, 64, 100000))
    if op == "pages":
        dt, cache = rng.choice([("f32", "f16"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f16", "e4m3")])
        R = _log(rng, 1, 64)
        high = _log(rng, 1, min(32768, 131072 // R))
        return dict(op=op, R=R, low=rng.randint(1, high), high=high, empty=rng.randint(0, R // 3), H=H, Hkv=Hkv,
                    hd=hd, dt=dt, cache=cache, page=rng.choice([8, 16, 32, 64, 128]))
    dt, kv = rng.choice([("f32", "f16"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
    B = _log(rng, 1, 16)
    Lq = _log(rng, 1, 4096 // B)
    Lk = _log(rng, 1, 4096)
    return dict(op=op, B=B, Lq=Lq, Lk=Lk, low=rng.randint(0, Lk), H=H, Hkv=Hkv, hd=hd, dt=dt, kv=kv)


def _spread(n, low, high):
    """n lengths from low to high, evenly spread over the logarithm where that spans more than a factor of ten."""
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


def _plan_lengths(case):
    """(cached, new) of every request: idle ones first, then the prompts, then the ones with a single token."""
    R, P, I = case["R"], case["prompts"], case["idle"]
    cached = _spread(R, case["low"], case["high"])
    # the cached lengths in a fixed mixed order, so that prompts and idle requests have long and short ones
    step = next(s for s in range(R // 2 + 1, 2 * R + 2) if math.gcd(s, R) == 1)
    cached = [cached[(i * step) % R] for i in range(R)]
    new = [0] * I + [max(1, x) for x in _spread(P, 2, case["longest"])]
    return cached, (new + [1] * R)[:R]


def _page_lengths(case):
    R = case["R"]
    e = min(case["empty"], R - 1)
    return [0] * e + _spread(R - e, case["low"], case["high"])


def _cross_lengths(case):
    return _spread(case["B"], case["low"], case["Lk"])


def _pages(n, page):
    return -(-n // page)


def _sections(case):
    """Pairs of each axis: time gets what height, width and a fourth axis leave."""
    half, A = case["hd"] // 2, case["axes"]
    each = half * 5 // 16
    s = [half // A] * A if A == 2 or A == 4 else [each] * A
    s[0] = half - sum(s[1:])
    return s


def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _plan_lengths(case)
        n, pg = sum(new), case["page"]
        taken = sum(_pages(c + x, pg) - _pages(c, pg) for c, x in zip(cached, new))
        # lengths in; pages taken from the free list into the tables; totals, starts; slot, position and request
        # of every new token
        old = sum(1 for c, x in zip(cached, new) if x and c % pg)
        return {"bytes": 8 * case["R"] + 8 * taken + 4 * old + 4 * (2 * case["R"] + 1) + 12 * n, "flops": 2 * n}
    if op == "write":
        n, hd, s = case["n"] - case["skipped"], case["hd"], SIZE[case["dt"]]
        b = n * hd * (2 * case["H"] * s + 2 * case["Hkv"] * (s + SIZE[case["cache"]]))
        return {"bytes": b + 4 * n * case["axes"] + 4 * case["n"], "flops": 3 * n * hd * (case["H"] + case["Hkv"])}
    if op == "pages":
        L = _page_lengths(case)
        t, hd = sum(L), case["hd"]
        return {"bytes": 2 * t * case["Hkv"] * hd * SIZE[case["cache"]] +
                2 * case["R"] * case["H"] * hd * SIZE[case["dt"]] + 4 * sum(_pages(x, case["page"]) for x in L),
                "flops": 4 * t * case["H"] * hd}
    L = _cross_lengths(case)
    hd = case["hd"]
    return {"bytes": 2 * sum(L) * case["Hkv"] * hd * SIZE[case["kv"]] +
            2 * case["B"] * case["Lq"] * case["H"] * hd * SIZE[case["dt"]],
            "flops": 4 * sum(L) * case["Lq"] * case["H"] * hd}


# ------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)

    def normal(*shape, dt="f32", scale=1.0):
        x = torch.empty(*shape, dtype=torch.float16 if dt == "e4m3" else DT[dt], device="cuda")
        x.normal_(0.0, scale, generator=g)
        return x.to(DT[dt])

    def shuffled(v):
        return [v[i] for i in torch.randperm(len(v), generator=h).tolist()]

    op = case["op"]
    st = dict(case=case, op=op)
    if op == "plan":
        pg, R = case["page"], case["R"]
        cached, new = _plan_lengths(case)
        order = torch.randperm(R, generator=h).tolist()
        cached, new = [cached[i] for i in order], [new[i] for i in order]
        n = sum(new)
        held = sum(_pages(c, pg) for c in cached)
        taken = sum(_pages(c + x, pg) - _pages(c, pg) for c, x in zip(cached, new))
        ids = torch.randperm(held + taken + 37, generator=h).to(torch.int32)
        width = max(1, max(_pages(c + x, pg) for c, x in zip(cached, new))) + 3
        table = torch.full((R, width), -1, dtype=torch.int32)
        owned = torch.arange(width)[None, :] < torch.tensor([_pages(c, pg) for c in cached])[:, None]
        table[owned] = ids[:held]
        rows = n + 29                                   # the step's fixed capacity of new tokens
        st.update(len=_ints(cached), new=_ints(new), free=ids[held:].cuda(), table=table.cuda(), rows=rows, page=pg,
                  total=torch.empty(R, dtype=torch.int32, device="cuda"),
                  start=torch.empty(R + 1, dtype=torch.int32, device="cuda"),
                  slot=torch.empty(rows, dtype=torch.int32, device="cuda"),
                  pos=torch.empty(rows, dtype=torch.int32, device="cuda"),
                  req=torch.empty(rows, dtype=torch.int32, device="cuda"),
                  info=torch.empty(4, dtype=torch.int32, device="cuda"))
    elif op == "write":
        n, H, Hkv, hd, pg = case["n"], case["H"], case["Hkv"], case["hd"], case["page"]
        qkv = normal(n, (H + 2 * Hkv) * hd, dt=case["dt"])
        n_pages = _pages(n, pg) + 5
        slot = torch.randperm(n_pages * pg, generator=h)[:n].to(torch.int32)
        slot[torch.randperm(n, generator=h)[:case["skipped"]]] = -1
        pos = torch.randint(0, case["far"], (case["axes"], n), generator=h).to(torch.int32)
        st.update(qkv=qkv, q=qkv[:, :H * hd], k=qkv[:, H * hd:(H + Hkv) * hd], v=qkv[:, (H + Hkv) * hd:],
                  slot=slot.cuda(), pos=pos.cuda(), sections=_sections(case),
                  qout=torch.zeros(n, H * hd, dtype=DT[case["dt"]], device="cuda"),
                  kc=torch.zeros(n_pages, Hkv, pg, hd, dtype=DT[case["cache"]], device="cuda"),
                  vc=torch.zeros(n_pages, Hkv, pg, hd, dtype=DT[case["cache"]], device="cuda"))
        if own:
            import autoregressive_speech_token_gb300 as sd
            st["rope"] = sd.sd_rope_init(hd, case["theta"], st["sections"], case["interleaved"])
            st["cache"] = sd.Pages.of(st["kc"], st["vc"])
            st["dtype"] = sd.DTYPES[case["dt"]]
    elif op == "pages":
        R, H, Hkv, hd, pg = case["R"], case["H"], case["Hkv"], case["hd"], case["page"]
        L = shuffled(_page_lengths(case))
        held = sum(_pages(x, pg) for x in L)
        ids = torch.randperm(held + 11, generator=h).to(torch.int32)
        width = max(1, max(_pages(x, pg) for x in L)) + 1
        table = torch.full((R, width), -1, dtype=torch.int32)
        owned = torch.arange(width)[None, :] < torch.tensor([_pages(x, pg) for x in L])[:, None]
        table[owned] = ids[:held]
        st.update(q=normal(R, H, hd, dt=case["dt"]), kc=normal(held + 11, Hkv, pg, hd, dt=case["cache"]),
                  vc=normal(held + 11, Hkv, pg, hd, dt=case["cache"]), table=table.cuda(), len=_ints(L),
                  scale=1.0 / math.sqrt(hd), out=torch.empty(R, H, hd, dtype=DT[case["dt"]], device="cuda"),
                  ks=None, vs=None)
        if case["cache"] == "e4m3":
            st["ks"] = torch.rand(Hkv, generator=g, device="cuda") * 0.5 + 0.75
            st["vs"] = torch.rand(Hkv, generator=g, device="cuda") * 0.5 + 0.75
        if own:
            import autoregressive_speech_token_gb300 as sd
            st["cache"] = sd.Pages.of(st["kc"], st["vc"], st["ks"], st["vs"])
            st["ws"] = sd.AttnWorkspace()
            st["dtype"] = sd.DTYPES[case["dt"]]
    else:
        B, Lq, Lk, H, Hkv, hd = (case[x] for x in ("B", "Lq", "Lk", "H", "Hkv", "hd"))
        st.update(q=normal(B, Lq, H, hd, dt=case["dt"]), k=normal(B, Lk, Hkv, hd, dt=case["kv"]),
                  v=normal(B, Lk, Hkv, hd, dt=case["kv"]), len=_ints(shuffled(_cross_lengths(case))),
                  scale=1.0 / math.sqrt(hd), out=torch.empty(B, Lq, H, hd, dtype=DT[case["dt"]], device="cuda"))
        if own:
            import autoregressive_speech_token_gb300 as sd
            st["states"] = sd.States.of(st["k"], st["v"], st["len"])
            st["ws"] = sd.AttnWorkspace()
            st["dtype"] = sd.DTYPES[case["dt"]]
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _own[st["op"]](st) if own else _plain[st["op"]](st)


def _plain_plan(st):
    ln, new, pg, rows = st["len"].long(), st["new"].long(), st["page"], st["rows"]
    table = st["table"]
    R, width = table.shape
    start = torch.zeros(R + 1, dtype=torch.int64, device=ln.device)
    start[1:] = torch.cumsum(new, 0)
    total = ln + new
    before, after = (ln + pg - 1) // pg, (total + pg - 1) // pg
    first = torch.cumsum(after - before, 0) - (after - before)
    col = torch.arange(width, device=ln.device)[None, :]
    fresh = (col >= before[:, None]) & (col < after[:, None])
    take = first[:, None] + col - before[:, None]
    table = torch.where(fresh, st["free"][take.clamp(0, st["free"].numel() - 1)], table)
    i = torch.arange(rows, device=ln.device)
    live = i < start[R]
    r = torch.searchsorted(start[1:], i, right=True).clamp(max=R - 1)
    p = ln[r] + i - start[r]
    page = table[r, (p // pg).clamp(0, width - 1)].long()
    slot = torch.where(live, page * pg + p % pg, -1)
    info = torch.stack([start[R], (after - before).sum(), torch.zeros_like(start[R]), total.max()])
    return [x.to(torch.int32) for x in (table, total, start, slot, torch.where(live, p, 0),
                                        torch.where(live, r, -1), info)]


def _axes(case):
    """Axis of each pair."""
    left, A, out = list(_sections(case)), case["axes"], []
    if not case["interleaved"]:
        return [a for a in range(A) for _ in range(left[a])]
    a = 0
    while len(out) < case["hd"] // 2:
        if left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % A
    return out


def _plain_write(st):
    c = st["case"]
    n, H, Hkv, hd, pg = c["n"], c["H"], c["Hkv"], c["hd"], c["page"]
    half = hd // 2
    ax = torch.tensor(_axes(c), device="cuda")
    freq = c["theta"] ** (-torch.arange(half, dtype=torch.float64, device="cuda") * 2 / hd)
    angle = st["pos"][ax].double().T * freq                       # [n][half], 64 bits: far positions
    cs, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x, heads):
        x = x.float().reshape(n, heads, hd)
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cs - b * sn, a * sn + b * cs], -1)

    live = torch.nonzero(st["slot"] >= 0)[:, 0]
    slot = st["slot"][live].long()
    st["qout"][live] = turn(st["q"], H).reshape(n, H * hd)[live].to(st["qout"].dtype)
    st["kc"][slot // pg, :, slot % pg] = turn(st["k"], Hkv)[live].to(st["kc"].dtype)
    st["vc"][slot // pg, :, slot % pg] = st["v"].reshape(n, Hkv, hd)[live].float().to(st["vc"].dtype)
    return st["qout"], st["kc"], st["vc"]


def _attend(q, k, v, live, scale):
    """q [B][Hkv][M][hd], k / v [B][Hkv][L][hd] in 32 bits, live [B][L]: softmax over the live positions."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = s.masked_fill_(~live[:, None, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    den = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(den == 0, torch.ones_like(den), den)


def _plain_pages(st):
    c, table = st["case"], st["table"].long().clamp(min=0)
    R, H, Hkv, hd = c["R"], c["H"], c["Hkv"], c["hd"]

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
    o = _attend(st["q"].float().reshape(R, Hkv, H // Hkv, hd), k, v, live, st["scale"])
    st["out"].copy_(o.reshape(R, H, hd))
    return st["out"]


def _plain_cross(st):
    c = st["case"]
    B, Lq, Lk, H, Hkv, hd = (c[x] for x in ("B", "Lq", "Lk", "H", "Hkv", "hd"))
    G = H // Hkv
    q = st["q"].float().reshape(B, Lq, Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Lq * G, hd)
    k, v = st["k"].float().transpose(1, 2), st["v"].float().transpose(1, 2)
    live = torch.arange(Lk, device="cuda")[None, :] < st["len"][:, None]
    o = _attend(q, k, v, live, st["scale"])
    st["out"].copy_(o.reshape(B, Hkv, Lq, G, hd).permute(0, 2, 1, 3, 4).reshape(B, Lq, H, hd))
    return st["out"]


_plain = dict(plan=_plain_plan, write=_plain_write, pages=_plain_pages, cross=_plain_cross)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _own_plan(st):
    import autoregressive_speech_token_gb300 as sd
    R, width = st["table"].shape
    sd.sd_page_plan(st["len"], st["new"], R, st["free"], st["free"].numel(), st["page"], st["table"], width,
                    st["rows"], st["total"], st["start"], st["slot"], st["pos"], st["req"], st["info"], _stream())
    return [st[x] for x in ("table", "total", "start", "slot", "pos", "req", "info")]


def _own_write(st):
    import autoregressive_speech_token_gb300 as sd
    c, ld = st["case"], st["qkv"].stride(0)
    sd.sd_rope_write_pages(st["rope"], st["pos"], c["n"], st["slot"], c["n"], st["dtype"], st["q"], ld, st["qout"],
                           c["H"] * c["hd"], c["H"], st["k"], st["v"], ld, st["cache"], _stream())
    return st["qout"], st["kc"], st["vc"]


def _own_pages(st):
    import autoregressive_speech_token_gb300 as sd
    R, H, hd = st["q"].shape
    sd.sd_attend_pages(st["ws"], st["cache"], st["table"], st["table"].shape[1], st["len"], R, st["dtype"], st["q"],
                       H * hd, H, st["scale"], st["out"], H * hd, None, _stream())
    return st["out"]


def _own_cross(st):
    import autoregressive_speech_token_gb300 as sd
    B, Lq, H, hd = st["q"].shape
    sd.sd_attend_cross(st["ws"], st["states"], st["dtype"], st["q"], Lq * H * hd, H * hd, Lq, H, st["scale"],
                       st["out"], Lq * H * hd, H * hd, None, _stream())
    return st["out"]


_own = dict(plan=_own_plan, write=_own_write, pages=_own_pages, cross=_own_cross)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(st)
    if op == "write":
        return _exact_write(st)
    if op == "pages":
        return _exact_pages(st)
    return _exact_cross(st)


def _exact_plan(st):
    pg, rows = st["page"], st["rows"]
    ln, new, free = (st[x].cpu().numpy().astype(np.int64) for x in ("len", "new", "free"))
    table = st["table"].cpu().numpy().copy()
    slot = np.full(rows, -1, np.int64)
    pos = np.zeros(rows, np.int64)
    req = np.full(rows, -1, np.int64)
    start = [0]
    used = 0
    for r in range(len(ln)):
        a, b = int(ln[r]), int(ln[r] + new[r])
        for page in range(-(-a // pg), -(-b // pg)):
            table[r, page] = free[used]
            used += 1
        at = start[-1]
        where = np.arange(a, b)
        slot[at:at + b - a] = table[r, where // pg].astype(np.int64) * pg + where % pg
        pos[at:at + b - a] = where
        req[at:at + b - a] = r
        start.append(at + b - a)
    info = [start[-1], used, 0, int((ln + new).max())]
    return [torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
            for x in (table, ln + new, start, slot, pos, req, info)]


def _exact_write(st):
    c = st["case"]
    n, H, Hkv, hd, pg = c["n"], c["H"], c["Hkv"], c["hd"], c["page"]
    pos = st["pos"].cpu().numpy().astype(np.float64)
    axis = _axes(c)
    z = np.empty((n, hd // 2), np.complex128)                     # a pair is a complex number, a position its turn
    for i in range(hd // 2):
        z[:, i] = np.exp(1j * pos[axis[i]] * c["theta"] ** (-2.0 * i / hd))
    z = torch.from_numpy(z).cuda()[:, None, :]

    def turn(x, heads):
        x = x.double().reshape(n, heads, 2, hd // 2)
        y = torch.complex(x[:, :, 0].contiguous(), x[:, :, 1].contiguous()) * z
        return torch.cat([y.real, y.imag], -1)

    live = st["slot"] >= 0
    s = st["slot"][live].long()
    q = torch.where(live[:, None], turn(st["q"], H).reshape(n, H * hd), st["qout"].double())
    out = [q]
    for pool, rows in ((st["kc"], turn(st["k"], Hkv)), (st["vc"], st["v"].double().reshape(n, Hkv, hd))):
        flat = pool.double().transpose(1, 2).reshape(-1, Hkv, hd).contiguous()
        flat[s] = rows[live]
        out.append(flat.reshape(pool.shape[0], pg, Hkv, hd).transpose(1, 2))
    return out


def _exact_rows(q, k, v, scale):
    """q [Hkv][M][hd], k / v [L][Hkv][hd] in 64 bits."""
    s = torch.einsum("gmd,lgd->gml", q, k) * scale
    return torch.einsum("gml,lgd->gmd", torch.softmax(s, -1), v)


def _exact_pages(st):
    c = st["case"]
    R, H, Hkv, hd, pg = c["R"], c["H"], c["Hkv"], c["hd"], c["page"]
    out = torch.zeros(R, H, hd, dtype=torch.float64, device="cuda")
    for r, n in enumerate(st["len"].tolist()):
        if n == 0:
            continue
        ids = st["table"][r, :_pages(n, pg)].tolist()

        def rows(pool, scale):
            x = torch.cat([pool[i].double().transpose(0, 1) for i in ids])[:n]
            return x if scale is None else x * scale.double()[None, :, None]

        o = _exact_rows(st["q"][r].double().reshape(Hkv, H // Hkv, hd), rows(st["kc"], st["ks"]),
                        rows(st["vc"], st["vs"]), st["scale"])
        out[r] = o.reshape(H, hd)
    return out


def _exact_cross(st):
    c = st["case"]
    B, Lq, H, Hkv, hd = (c[x] for x in ("B", "Lq", "H", "Hkv", "hd"))
    G = H // Hkv
    out = torch.zeros(B, Lq, H, hd, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["len"].tolist()):
        if n == 0:
            continue
        for h in range(H):
            g = h // G
            for a in range(0, Lq, 4096):
                o = _exact_rows(st["q"][b, a:a + 4096, h].double()[None], st["k"][b, :n, g:g + 1].double(),
                                st["v"][b, :n, g:g + 1].double(), st["scale"])
                out[b, a:a + 4096, h] = o[0]
    return out
