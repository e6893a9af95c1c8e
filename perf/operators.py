"""Timed cases of the paged latent cache: append, attention of new rows over the
cache (whole, windowed with sinks, and with the attention weights accumulated),
and eviction by accumulated weight.

A case names an operator and its sizes.  `run` computes it either through the
package (`own` true) or in plain torch operations, in fp32, rounded once at the
end.  The lengths of a batch follow from the case alone, the values from the
seed.
"""
import math
import random

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# op            append | attend | mass (attend + accumulate the weights) | evict
# heads, rank   query heads sharing one latent K = V row of width rank
# page          slots of a page
# batch         users
# len_lo/hi     cached events per user, the new ones included (uniform)
# new_lo/hi     new events per user (uniform, at most the length)
# cand          query tokens per user, which see every event
# window, sink  0 = the whole history; otherwise the last `window` events and the first `sink`
# budget, recent  eviction: events kept per user, and the newest that always stay
_BASE = dict(op="attend", dtype="bf16", heads=4, rank=128, page=64, batch=1, len_lo=1, len_hi=1,
             new_lo=0, new_hi=0, cand=0, window=0, sink=0, budget=0, recent=0)


def _case(**kw):
    c = dict(_BASE)
    c.update(kw)
    return c


def listed():
    return [
        # a burst of a few new events of one user, fp32: pure latency
        _case(name="append_burst_fp32", op="append", dtype="fp32", heads=2, rank=32, page=16,
              batch=1, len_lo=60, len_hi=60, new_lo=5, new_hi=5),
        # the histories of a whole batch enter the cache at once
        _case(name="append_histories", op="append", batch=256, len_lo=100, len_hi=400,
              new_lo=100, new_hi=400),
        # one new event of one user over its history: the smallest request
        _case(name="attend_one_token", batch=1, len_lo=399, len_hi=399, new_lo=1, new_hi=1),
        # one new event for each of many users with long histories
        _case(name="attend_tokens_long", heads=8, rank=256, batch=64, len_lo=2000, len_hi=8000,
              new_lo=1, new_hi=1),
        # an online request: a few new events and 64 candidates per user
        _case(name="attend_candidates", batch=256, len_lo=100, len_hi=400, new_lo=0, new_hi=16,
              cand=64),
        # a user model is brought up to date with a long chunk of new events
        _case(name="attend_chunk", heads=8, rank=256, batch=32, len_lo=900, len_hi=1600,
              new_lo=500, new_hi=800),
        # one new event per user, windowed, fp32 on a narrow model
        _case(name="window_tokens_fp32", dtype="fp32", heads=2, rank=32, page=32, batch=64,
              len_lo=500, len_hi=4000, new_lo=1, new_hi=1, window=256, sink=4),
        # a long history streams in behind a window, odd sizes
        _case(name="window_chunk", batch=24, len_lo=1000, len_hi=4000, new_lo=333, new_hi=777,
              window=401, sink=17, page=128),
        # one new event per user; its weights decide what is evicted later
        _case(name="mass_tokens", op="mass", heads=8, rank=256, batch=128, len_lo=800,
              len_hi=1600, new_lo=1, new_hi=1),
        # candidates of an online request vote on the events
        _case(name="mass_candidates", op="mass", batch=256, len_lo=100, len_hi=400, new_lo=0,
              new_hi=16, cand=64),
        # a handful of users pruned, fp32
        _case(name="evict_few_fp32", op="evict", dtype="fp32", heads=2, rank=32, page=16, batch=4,
              len_lo=150, len_hi=400, budget=128, recent=32, sink=4),
        # a whole batch pruned to a third
        _case(name="evict_batch", op="evict", heads=8, rank=256, batch=256, len_lo=700,
              len_hi=1600, budget=512, recent=128, sink=4),
    ]


_MOST = {}


def _most():
    if not _MOST:
        for c in listed():
            for k, v in work(c).items():
                _MOST[k] = max(_MOST.get(k, 0), v)
    return _MOST


def _log(rng, lo, hi):
    return int(round(2 ** rng.uniform(math.log2(lo), math.log2(hi))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "mass", "mass", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    rank = rng.choice([32, 64, 128] if dtype == "fp32" else [64, 128, 128, 256])
    c = _case(op=op, dtype=dtype, rank=rank, heads=rng.choice([1, 2, 3, 4, 8]),
              page=rng.choice([16, 32, 64, 128]), batch=_log(rng, 1, 256))
    c["len_hi"] = _log(rng, 40, 6000)
    c["len_lo"] = rng.randint(c["len_hi"] // 3, c["len_hi"])
    if op == "append":
        c["new_hi"] = _log(rng, 1, c["len_hi"])
        c["new_lo"] = rng.randint(0 if c["batch"] > 8 else 1, c["new_hi"])
    elif op == "evict":
        c["budget"] = max(8, _log(rng, 8, c["len_hi"]))
        c["recent"] = rng.randint(0, c["budget"] // 2)
        c["sink"] = rng.randint(0, min(16, c["budget"] // 4))
    else:
        kind = rng.choice(["token", "cands", "chunk"])
        if kind == "token":
            c["new_lo"] = c["new_hi"] = 1
        elif kind == "cands":
            c["new_hi"], c["cand"] = rng.randint(0, 20), _log(rng, 1, 128)
        else:
            c["new_hi"] = _log(rng, 2, max(2, min(800, c["len_hi"])))
            c["new_lo"] = rng.randint(1, c["new_hi"])
        if rng.random() < 0.4:
            c["window"], c["sink"] = _log(rng, 1, 1000), rng.choice([0, 1, 4, 33])
    # no drawn case costs more than the largest listed one, also where the plain
    # form computes the scores that a window hides
    top = _most()
    pairs = (c["new_hi"] + c["cand"]) * c["heads"] if op in ("attend", "mass") else 0
    while c["batch"] > 1 and (any(v > 0.8 * top[k] for k, v in work(c).items())
                              or c["batch"] * pairs * c["len_hi"] > 5e8):
        c["batch"] //= 2
    while any(v > 0.8 * top[k] for k, v in work(c).items()):
        for k in ("len_lo", "len_hi", "new_lo", "new_hi"):
            c[k] = (c[k] + 1) // 2
    return c


def _sizes(case):
    """Per user: cached events (new ones included) and new events."""
    keys = sorted(k for k in case if k != "name")
    rng = random.Random(repr([(k, case[k]) for k in keys]))
    lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    news = [min(n, rng.randint(case["new_lo"], case["new_hi"])) for n in lens]
    return lens, news


def work(case):
    lens, news = _sizes(case)
    h, r, e = case["heads"], case["rank"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        # new rows read and written, their masses cleared, the gain
        return {"bytes": sum(news) * (2 * r * e + 4) + r * e, "flops": 4 * r * sum(news)}
    if case["op"] == "evict":
        kept = [min(n, case["budget"]) for n in lens]
        return {"bytes": 4 * sum(lens) + sum(kept) * (2 * r * e + 4 + 4), "flops": sum(lens)}
    W, S, cand = case["window"], case["sink"], case["cand"]
    flops = keys = rows = 0
    for n, m in zip(lens, news):
        rows += m + cand
        first = n - 1 if m == 0 else n - m            # the earliest position that asks
        seen = lambda p: p + 1 if W == 0 or p + 1 <= W else W + min(S, p + 1 - W)  # noqa: E731
        flops += 4 * r * h * (sum(seen(p) for p in range(n - m, n)) + cand * seen(n - 1))
        if m + cand:
            low = 0 if W == 0 else max(0, first - W + 1)
            keys += n - low + min(S, low)
    nbytes = keys * r * e + 2 * rows * h * r * e
    if case["op"] == "mass":
        nbytes += 8 * keys
    return {"bytes": nbytes, "flops": flops}


def _randn(gen, shape, dt):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    lens, news = _sizes(case)
    B, h, r, P = case["batch"], case["heads"], case["rank"], case["page"]
    npg = [-(-n // P) for n in lens]
    width = max(npg)
    src_pages = sum(npg) + 3
    kept_pages = [-(-min(n, case["budget"]) // P) for n in lens] if case["op"] == "evict" else []
    n_pages = src_pages + sum(kept_pages)

    def table(first, counts, total, width):
        ids = list(range(first, first + total))
        rng.shuffle(ids)
        t = torch.zeros((B, max(width, 1)), dtype=torch.int32)
        for u, n in enumerate(counts):
            t[u, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
        return t.cuda()

    st = {"case": case, "h": h, "r": r, "P": P, "src_pages": src_pages,
          "lengths": torch.tensor(lens, dtype=torch.int32).cuda(),
          "table": table(0, npg, src_pages, width),
          "mass": torch.zeros((n_pages, P), device="cuda")}
    off = [0]
    for m in news:
        off.append(off[-1] + m + (0 if case["op"] == "append" else case["cand"]))
    st["offsets"] = torch.tensor(off, dtype=torch.int64).cuda()
    rows = off[-1]
    if case["op"] == "append":
        st["pool"] = torch.zeros((n_pages, P, r), device="cuda", dtype=dt)
        # the projected latents before their norm
        st["x"] = _randn(gen, (rows, r), dt)
        st["gain"] = (1 + 0.1 * _randn(gen, (r,), torch.float32)).to(dt)
    else:
        # the latents are RMS-normalised rows
        st["pool"] = _randn(gen, (n_pages, P, r), dt)
    if case["op"] in ("attend", "mass"):
        # heads of different sharpness: scores of deviation 0.5 to 3
        sharp = torch.linspace(0.5, 3.0, h, device="cuda")[:, None]
        st["q"] = (_randn(gen, (rows, h, r), torch.float32) * sharp).to(dt)
        st["scale"] = r ** -0.5
        if case["op"] == "mass":
            st["mass"] = torch.rand((n_pages, P), generator=gen, device="cuda")
    if case["op"] == "evict":
        # heavy-tailed weights, an eighth of the events never looked at (ties)
        m = torch.exp(2 * _randn(gen, (n_pages, P), torch.float32))
        st["mass"] = m * (torch.rand((n_pages, P), generator=gen, device="cuda") > 0.125)
        st["pool"][src_pages:] = 0
        st["mass"][src_pages:] = 0
        st["dst"] = table(src_pages, kept_pages, sum(kept_pages), max(kept_pages))
        st["new_lengths"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        st["kept"] = torch.full((B, case["budget"]), -1, dtype=torch.int32, device="cuda")
    if case["op"] == "mass" or case["op"] == "attend":
        st["out"] = torch.empty((rows, h, r), device="cuda", dtype=dt)
        st["lse"] = torch.empty((rows, h), device="cuda")
    st["max_rows"] = max(rows, 1)
    st["cache"] = None
    if own:
        from latent_attention_jagged_b200 import LatentCache
        st["cache"] = LatentCache(st["pool"], heads=h, mass=st["mass"], max_batch=B,
                                  max_rows=st["max_rows"], max_pages=max(width, 1))
    return st


def run(st):
    op = st["case"]["op"]
    if op == "append":
        return _append(st)
    if op == "evict":
        return _evict(st)
    return _attend(st, op == "mass")


def _append(st):
    if own:
        st["cache"].append(st["x"], st["offsets"], st["table"], st["lengths"], gain=st["gain"],
                           eps=EPS)
        return {"pool": st["pool"], "mass": st["mass"]}
    x = st["x"].float()
    c = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * st["gain"].float()
    off, lens, P = st["offsets"], st["lengths"].long(), st["P"]
    row = torch.arange(x.shape[0], device=x.device)
    user = torch.searchsorted(off, row, right=True) - 1
    slot = lens[user] - (off[user + 1] - row)
    page = st["table"].long()[user, slot // P]
    st["pool"][page, slot % P] = c.to(st["pool"].dtype)
    st["mass"][page, slot % P] = 0
    return {"pool": st["pool"], "mass": st["mass"]}


def _attend(st, accumulate):
    c = st["case"]
    if own:
        st["cache"].attend(st["q"], st["offsets"], st["table"], st["lengths"], n_cand=c["cand"],
                           scale=st["scale"], window=c["window"], n_sink=c["sink"],
                           out=st["out"], lse=st["lse"], accumulate=accumulate)
        outs = {"out": st["out"], "lse": st["lse"]}
        if accumulate:
            outs["mass"] = st["mass"]
        return outs
    q, off, P, h, r = st["q"], st["offsets"], st["P"], st["h"], st["r"]
    lens = st["lengths"].long()
    B, T = lens.shape[0], st["table"].shape[1] * P
    K = st["pool"][st["table"].long()].reshape(B, T, r).float()
    rows = off[1:] - off[:-1]
    R = int(st["case"]["new_hi"]) + c["cand"]
    j = torch.arange(R, device=q.device)
    have = j[None] < rows[:, None]                                        # [B, R]
    at = torch.where(have, off[:-1, None] + j[None], 0)
    Q = q[at].float()                                                    # [B, R, h, r]
    new = rows - c["cand"]
    pos = torch.where(j[None] < new[:, None], lens[:, None] - new[:, None] + j[None],
                      lens[:, None] - 1)                                 # [B, R]
    t = torch.arange(T, device=q.device)
    see = t[None, None] <= pos[:, :, None]
    if c["window"]:
        see = see & ((t > pos[:, :, None] - c["window"]) | (t < c["sink"]))
    see = (see & have[:, :, None]).repeat_interleave(h, dim=1)           # [B, R h, T]
    s = torch.matmul(Q.reshape(B, R * h, r), K.transpose(1, 2)) * st["scale"]
    s = torch.where(see, s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, 1.0)
    o = torch.matmul(p, torch.where((t[None] < lens[:, None])[:, :, None], K, 0.0))
    lse = (torch.log(l) + m).reshape(B, R, h)
    out, lout = st["out"], st["lse"]
    out[at[have]] = o.reshape(B, R, h, r)[have].to(out.dtype)
    lout[at[have]] = lse[have]
    if not accumulate:
        return {"out": out, "lse": lout}
    w = p.sum(1)                                                         # [B, T]
    cached = t[None] < lens[:, None]
    page = st["table"].long()[:, t // P]
    st["mass"][page[cached], (t % P).expand(B, T)[cached]] += w[cached]
    return {"out": out, "lse": lout, "mass": st["mass"]}


def _evict(st):
    c, P, first = st["case"], st["P"], st["src_pages"]
    if own:
        st["cache"].evict(st["table"], st["lengths"], budget=c["budget"], n_sink=c["sink"],
                          n_recent=c["recent"], dst_table=st["dst"],
                          new_lengths=st["new_lengths"], kept=st["kept"])
    else:
        lens = st["lengths"].long()
        B, T, K = lens.shape[0], st["table"].shape[1] * P, c["budget"]
        t = torch.arange(T, device=lens.device)
        cached = t[None] < lens[:, None]
        flat = st["mass"][st["table"].long()].reshape(B, T)
        stay = (t[None] < c["sink"]) | (t[None] >= lens[:, None] - c["recent"])
        key = torch.where(stay, float("inf"), flat)
        key = torch.where(cached, key, float("-inf"))
        order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :K]
        n = torch.clamp(lens, max=K)
        i = torch.arange(order.shape[1], device=lens.device)
        order = torch.where(i[None] < n[:, None], order, T)              # fillers sort last
        order = torch.sort(order, dim=1).values
        have = i[None] < n[:, None]
        u = torch.arange(B, device=lens.device)[:, None].expand_as(order)[have]
        s, d = order[have], i[None].expand_as(order)[have]
        sp, dp = st["table"].long()[u, s // P], st["dst"].long()[u, d // P]
        st["pool"][dp, d % P] = st["pool"][sp, s % P]
        st["mass"][dp, d % P] = st["mass"][sp, s % P]
        st["kept"][u, d] = s.int()
        st["new_lengths"].copy_(n.int())
    return {"pool": st["pool"][first:], "mass": st["mass"][first:], "kept": st["kept"],
            "new_lengths": st["new_lengths"]}


def exact(case, seed):
    """The definitions in 64 bits, user by user."""
    st = _prepared_for_exact(case, seed)
    lens, news = _sizes(case)
    table, P = st["table"].tolist(), case["page"]
    pool, mass = st["pool"].double(), st["mass"].double()
    off = st["offsets"].tolist()

    def places(u, slots, tab):
        slots = torch.as_tensor(slots, device="cuda")
        ids = torch.tensor(tab[u], device="cuda")[slots // P]
        return ids, slots % P

    if case["op"] == "append":
        g = st["gain"].double()
        for u in range(case["batch"]):
            if off[u + 1] > off[u]:
                x = st["x"][off[u]:off[u + 1]].double()
                at = places(u, list(range(lens[u] - news[u], lens[u])), table)
                pool[at] = x / torch.sqrt((x ** 2).mean(1, keepdim=True) + EPS) * g
                mass[at] = 0
        return {"pool": pool, "mass": mass}
    if case["op"] == "evict":
        kept, dst, K = st["kept"].cpu(), st["dst"].tolist(), case["budget"]
        for u, n in enumerate(lens):
            w = mass[places(u, list(range(n)), table)].tolist()
            stay = set(range(n)) if n <= K else \
                set(range(case["sink"])) | set(range(n - case["recent"], n))
            rest = sorted((t for t in range(n) if t not in stay), key=lambda t: (-w[t], t))
            slots = sorted(stay | set(rest[:max(0, min(n, K) - len(stay))]))
            kept[u, :len(slots)] = torch.tensor(slots, dtype=torch.int32)
            src, to = places(u, slots, table), places(u, list(range(len(slots))), dst)
            pool[to], mass[to] = pool[src], mass[src]
        first = st["src_pages"]
        return {"pool": pool[first:], "mass": mass[first:], "kept": kept,
                "new_lengths": torch.tensor([min(n, K) for n in lens])}
    out = torch.zeros_like(st["q"], dtype=torch.float64)
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for u in range(case["batch"]):
        a, b, n, m = off[u], off[u + 1], lens[u], news[u]
        if b == a:
            continue
        at = places(u, list(range(n)), table)
        c = pool[at]
        p = torch.tensor(list(range(n - m, n)) + [n - 1] * case["cand"], device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None]
        hidden = t > p
        if case["window"]:
            hidden |= (t <= p - case["window"]) & (t >= case["sink"])
        s = torch.einsum("ihr,tr->hit", st["q"][a:b].double(), c) * st["scale"]
        s = s.masked_fill(hidden, float("-inf"))
        lse[a:b] = torch.logsumexp(s, -1).T
        w = torch.softmax(s, -1)
        out[a:b] = torch.einsum("hit,tr->ihr", w, c)
        if case["op"] == "mass":
            mass[at] += w.sum((0, 1))
    res = {"out": out, "lse": lse}
    if case["op"] == "mass":
        res["mass"] = mass
    return res


def _prepared_for_exact(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was
