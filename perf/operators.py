"""What is measured of the paged 8-bit caches: the page plan, the quantising append, the 8-bit
indexer scores and the sparse attention over 8-bit latent rows, each in its plain form and
through the library's own entry points.

Cache layout (64 tokens to a page): a latent page is 64 rows of 592 bytes (576 e4m3 codes, the
row's fp32 scale, 12 bytes of padding); a key page is 64 x 128 e4m3 codes followed by the 64
keys' fp32 scales (8448 bytes). Scales are powers of two.
"""
import math
import random

import torch

own = False

PAGE = 64
LAT_ROW, LAT, VALUES = 592, 576, 512
KEY_PAGE, KEY = 8448, 128
HEADS = 32
F8 = torch.float8_e4m3fn


def listed():
    # `new`: rows (newest tokens) of each sequence; `lo`..`hi`: cached lengths, those rows included.
    return [
        # one decode step's bookkeeping of a serving batch, and a scheduler step that mixes long prompts with decodes
        dict(name="plan_decode", op="plan", n_seq=64, lo=16384, hi=32768, fresh=1, pad=0, mix=1),
        dict(name="plan_mixed", op="plan", n_seq=1000, lo=0, hi=9001, fresh=2500, pad=77, mix=2),
        # the new tokens of a decode step, and of a whole prompt
        dict(name="append_decode", op="append", n_rows=64, n_sub=2, pages=2048, gap=0),
        dict(name="append_prompt", op="append", n_rows=16384, n_sub=2, pages=300, gap=64),
        # latency of a single token; the long-context batch; ragged serving lengths; a prompt's chunk of rows
        dict(name="scores_b1_8k", op="scores", n_seq=1, lo=8192, hi=8192, new=1, ragged=False, topk=2048, init=16, local=1024, pad=0, mix=3),
        dict(name="scores_b16_128k", op="scores", n_seq=16, lo=131072, hi=131072, new=1, ragged=False, topk=2048, init=16, local=1024, pad=0, mix=4),
        dict(name="scores_b64_ragged", op="scores", n_seq=64, lo=16384, hi=32768, new=1, ragged=False, topk=2048, init=16, local=1024, pad=3, mix=5),
        dict(name="scores_rows4096_16k", op="scores", n_seq=1, lo=16384, hi=16384, new=4096, ragged=False, topk=2048, init=16, local=1024, pad=0, mix=6),
        # the same for the attention; the ragged batch holds rows shorter than the selection (dense rows)
        dict(name="mla_b1_8k", op="mla", n_seq=1, lo=8192, hi=8192, new=1, ragged=False, topk=2048, n_sub=2, pad=0, mix=7),
        dict(name="mla_b16_128k", op="mla", n_seq=16, lo=131072, hi=131072, new=1, ragged=False, topk=2048, n_sub=2, pad=0, mix=8),
        dict(name="mla_b64_ragged", op="mla", n_seq=64, lo=301, hi=9000, new=3, ragged=True, topk=2048, n_sub=1, pad=5, mix=9),
        dict(name="mla_rows2048_16k", op="mla", n_seq=1, lo=16384, hi=16384, new=2048, ragged=False, topk=2048, n_sub=2, pad=0, mix=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, mix = rng.choice(["plan", "append", "scores", "scores", "mla", "mla"]), rng.randrange(1 << 30)
    if op == "plan":
        n_seq = _log(rng, 1, 4096)
        return dict(op=op, n_seq=n_seq, lo=rng.choice([0, 0, 100]), hi=_log(rng, 200, 40000), fresh=_log(rng, 1, max(1, min(8000, 2500000 // n_seq))), pad=rng.choice([0, 1, 130]), mix=mix)
    if op == "append":
        n_rows = _log(rng, 1, 16384)
        return dict(op=op, n_rows=n_rows, n_sub=rng.choice([1, 2]), pages=-(-n_rows // PAGE) + _log(rng, 1, 300), gap=rng.choice([0, 8, 64]))
    topk = rng.choice([2048, 2048, 2048, 1500, 511, 64])
    many = rng.random() < 0.4  # many rows of few sequences, or few rows of many
    n_sub = rng.choice([1, 2]) if op == "mla" else 1
    hi = _log(rng, 1, 40000 if many else 200000)
    lo = rng.choice([hi, max(1, hi // 2), 1])
    new = _log(rng, 16, 2048) if many else rng.choice([1, 1, 2, 4])
    n_seq = _log(rng, 1, 6 if many else 96)
    if op == "scores":
        n_seq = max(1, min(n_seq, 4000000 // hi, 60000000 // (hi * new)))
        new = max(1, min(new, 60000000 // (hi * n_seq)))
        return dict(op=op, n_seq=n_seq, lo=lo, hi=hi, new=new, ragged=rng.random() < 0.5, topk=topk, init=min(16, topk // 4), local=min(1024, topk // 2), pad=rng.choice([0, 0, 7]), mix=mix)
    n_seq = max(1, min(n_seq, 1500000 // hi, 50000000 // (hi * new)))
    new = max(1, min(new, 2048 // (n_seq * n_sub) * 2, 50000000 // (hi * n_seq)))
    return dict(op=op, n_seq=n_seq, lo=lo, hi=hi, new=new, ragged=rng.random() < 0.5, topk=topk, n_sub=n_sub, pad=rng.choice([0, 0, 5]), mix=mix)


# ---- the geometry that a case stands for


def _requests(case):
    r = random.Random(case["mix"])
    cached = [r.randint(case["lo"], case["hi"]) for _ in range(case["n_seq"])]
    fresh = [1 if case["fresh"] == 1 else r.choice([0, 1, 1, 1, r.randint(1, case["fresh"])]) for _ in cached]
    return cached, fresh


def _taken(cached, fresh):
    return sum(-(-(c + f) // PAGE) - -(-c // PAGE) for c, f in zip(cached, fresh))


def _geometry(case):
    """Lengths, and (sequence, position) of each row: the newest tokens of each sequence."""
    r = random.Random(case["mix"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["n_seq"])]
    new = [min(n, r.randint(1, case["new"]) if case["ragged"] else case["new"]) for n in lens]
    return lens, [(s, n - k + i) for s, (n, k) in enumerate(zip(lens, new)) for i in range(k)]


def work(case):
    if case["op"] == "plan":
        cached, fresh = _requests(case)
        taken = _taken(cached, fresh)
        return {"bytes": 8 * case["n_seq"] + 8 * taken + 12 * (sum(fresh) + case["pad"]), "flops": 0}
    if case["op"] == "append":
        return {"bytes": case["n_rows"] * (4 + case["n_sub"] * (2 * LAT + LAT + 4) + 2 * KEY + KEY + 4), "flops": 0}
    lens, rows = _geometry(case)
    if case["op"] == "scores":
        pairs = sum(p + 1 for _, p in rows)
        return {"bytes": sum(lens) * (KEY + 4) + len(rows) * (2 * HEADS * KEY + 4 * HEADS) + 4 * pairs, "flops": 2 * HEADS * KEY * pairs}
    picks = sum(min(p + 1, case["topk"]) for _, p in rows)
    keys = min(picks, sum(lens)) * case["n_sub"]  # rows of one sequence share keys: each read once
    out = len(rows) * (2 * HEADS * (LAT + VALUES) + 4 * HEADS)
    return {"bytes": keys * (LAT + 4) + 4 * picks + case["n_sub"] * out, "flops": 2 * HEADS * (LAT + VALUES) * picks * case["n_sub"]}


# ---- inputs


def _quant(x):
    """Codes and power-of-two scale of each row (last dim) of fp32 x: x / s in e4m3, amax <= 448 s."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = torch.where(m > 0, torch.where(m <= 0.875, e - 9, e - 8), torch.zeros_like(e)).clamp(min=-126)
    return torch.ldexp(x, -e).to(F8), torch.ldexp(torch.ones_like(m), e)


def _latent_pages(n_pages, g):
    pool = torch.zeros(n_pages * PAGE, LAT_ROW, dtype=torch.uint8, device="cuda")
    x = torch.empty(n_pages * PAGE, LAT, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    codes, scale = _quant(x.float())
    pool[:, :LAT] = codes.view(torch.uint8)
    pool[:, LAT:LAT + 4] = scale.view(torch.uint8)
    return pool.view(n_pages, PAGE, LAT_ROW)


def _key_pages(n_pages, g):
    x = torch.empty(n_pages * PAGE, KEY, dtype=torch.float32, device="cuda").normal_(generator=g)
    x = (x / x.square().mean(-1, keepdim=True).sqrt()).bfloat16()
    codes, scale = _quant(x.float())
    pool = torch.empty(n_pages, KEY_PAGE, dtype=torch.uint8, device="cuda")
    pool[:, :PAGE * KEY] = codes.view(torch.uint8).view(n_pages, PAGE * KEY)
    pool[:, PAGE * KEY:] = scale.view(n_pages, PAGE).view(torch.uint8)
    return pool


def _tables(lens, g):
    """Block tables over a pool a little larger than the sequences need, pages in no order."""
    per = [-(-n // PAGE) for n in lens]
    order = torch.randperm(sum(per) + 5, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(per):
        table[s, :n] = order[at:at + n]
        at += n
    return table, order.numel()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"op": case["op"]}
    if case["op"] == "plan":
        cached, fresh = _requests(case)
        taken, width = _taken(cached, fresh), -(-(case["hi"] + case["fresh"]) // PAGE)
        owned = torch.tensor([-(-c // PAGE) for c in cached], **i32)
        n_pages = int(owned.sum()) + taken + 9
        order = torch.randperm(n_pages, generator=g, device="cuda").int()
        cols = torch.arange(width, **i32)
        first = owned.cumsum(0) - owned
        at = (first[:, None] + cols[None]).clamp(max=n_pages - 1)
        table = torch.where(cols[None] < owned[:, None], order[at.long()], torch.full_like(at, -1).int())
        s |= {"cached": torch.tensor(cached, **i32), "fresh": torch.tensor(fresh, **i32), "free": order[int(owned.sum()):].contiguous(), "table": table.contiguous(), "cap": sum(fresh) + case["pad"]}
        n = s["cap"]
        s |= {"seq": torch.empty(n, **i32), "pos": torch.empty(n, **i32), "slot": torch.empty(n, **i32), "totals": torch.empty(2, **i32)}
        return s
    if case["op"] == "append":
        n, wide = case["n_rows"], LAT + case["gap"]
        size = torch.exp2(torch.randint(-3, 4, (n, 1), generator=g, device="cuda").float())
        # the projection's output holds the latent next to other columns: rows are `wide` apart
        s["latent"] = [(torch.randn(n, wide, generator=g, device="cuda") * size).bfloat16()[:, :LAT] for _ in range(case["n_sub"])]
        k = torch.randn(n, KEY, generator=g, device="cuda")
        s["k"] = (k / k.square().mean(-1, keepdim=True).sqrt()).bfloat16()
        s["slot"] = torch.randperm(case["pages"] * PAGE, generator=g, device="cuda")[:n].int()
        s["slot"][5::97] = -1  # a padded batch: these rows are not kept
        s["latent_pages"] = [torch.zeros(case["pages"], PAGE, LAT_ROW, dtype=torch.uint8, device="cuda") for _ in range(case["n_sub"])]
        s["key_pages"] = torch.zeros(case["pages"], KEY_PAGE, dtype=torch.uint8, device="cuda")
        return s
    lens, rows = _geometry(case)
    n = len(rows) + case["pad"]
    s["seq"] = torch.tensor([r[0] for r in rows] + [-1] * case["pad"], **i32)
    s["pos"] = torch.tensor([r[1] for r in rows] + [-1] * case["pad"], **i32)
    s["table"], n_pages = _tables(lens, g)
    s["max_len"], s["topk"] = max(lens), case["topk"]
    if case["op"] == "scores":
        s["init"], s["local"] = case["init"], case["local"]
        s["q"] = torch.randn(n, HEADS, KEY, generator=g, device="cuda").bfloat16()
        s["w"] = torch.randn(n, HEADS, generator=g, device="cuda") * 0.03125 ** 0.5
        s["key_pages"] = _key_pages(n_pages, g)
        s["scores"] = torch.full((n, s["max_len"]), -math.inf, device="cuda")
        # the row's place among its sequence's rows (the plain form sets them side by side)
        first = {}
        rank = [p - first.setdefault(b, p) for b, p in rows]
        s["rank"], s["most"] = torch.tensor(rank + [0] * case["pad"], device="cuda"), max(rank) + 1
        return s
    s["n_sub"] = case["n_sub"]
    s["q"] = [torch.randn(n, HEADS, LAT, generator=g, device="cuda").bfloat16() for _ in range(case["n_sub"])]
    s["latent_pages"] = [_latent_pages(n_pages, g) for _ in range(case["n_sub"])]
    # a selection as the top-k leaves it: distinct visible keys, all of them where they are few, -1 behind them
    r = torch.rand(n, s["max_len"], generator=g, device="cuda")
    r.masked_fill_(torch.arange(s["max_len"], device="cuda")[None] > s["pos"][:, None], -1.0)
    k = min(s["topk"], s["max_len"])
    best, at = r.topk(k, dim=1)
    s["idx"] = torch.full((n, s["topk"]), -1, **i32)
    s["idx"][:, :k] = torch.where(best >= 0, at, torch.full_like(at, -1)).int()
    s["count"] = (s["pos"] + 1).clamp(max=s["topk"])
    s["out"] = [torch.zeros(n, HEADS, VALUES, dtype=torch.bfloat16, device="cuda") for _ in range(case["n_sub"])]
    s["lse"] = [torch.zeros(n, HEADS, device="cuda") for _ in range(case["n_sub"])]
    return s


# ---- one pass


def run(s):
    return {"plan": _run_plan, "append": _run_append, "scores": _run_scores, "mla": _run_mla}[s["op"]](s)


def _run_plan(s):
    if own:
        from sparse_attention_03_b200 import lsa

        if "call" not in s:  # marshalled once, as a serving loop with fixed buffers does
            s["call"] = lsa.page_plan(s["cached"], s["fresh"], s["free"], s["table"], s["seq"], s["pos"], s["slot"], s["totals"], bind=True)
        s["call"]()
        return {k: s[k] for k in ("table", "seq", "pos", "slot", "totals")}
    cached, fresh, table = s["cached"].long(), s["fresh"].long(), s["table"].clone()
    owned = (cached + PAGE - 1) // PAGE
    needed = (cached + fresh + PAGE - 1) // PAGE - owned
    upto = needed.cumsum(0)
    cols = torch.arange(table.shape[1], device=table.device)[None]
    mine = (cols >= owned[:, None]) & (cols < (owned + needed)[:, None])
    which = (upto - needed - owned)[:, None] + cols
    table = torch.where(mine, s["free"][which.clamp(0, s["free"].numel() - 1)], table)
    ends = fresh.cumsum(0)
    row = torch.arange(s["cap"], device=table.device)
    seq = torch.searchsorted(ends, row, right=True)
    real = seq < ends.numel()
    at = seq.clamp(max=ends.numel() - 1)
    pos = cached[at] + row - (ends - fresh)[at]
    slot = table[at, (pos // PAGE).clamp(max=table.shape[1] - 1)] * PAGE + pos % PAGE
    hide = lambda x: torch.where(real, x, torch.full_like(x, -1)).int()  # noqa: E731
    return {"table": table, "seq": hide(seq), "pos": hide(pos), "slot": hide(slot), "totals": torch.stack([ends[-1], upto[-1]]).int()}


def _seen(latent_pages, key_pages):
    """The caches as the values they stand for: e4m3 codes and their scales."""
    rows = [p.view(-1, LAT_ROW) for p in latent_pages]
    return {
        "latent": [r[:, :LAT].view(F8) for r in rows],
        "latent_scale": [r.view(torch.float32)[:, LAT // 4] for r in rows],
        "key": key_pages[:, :PAGE * KEY].view(F8),
        "key_scale": key_pages.view(torch.float32)[:, PAGE * KEY // 4:],
    }


def _run_append(s):
    if own:
        from sparse_attention_03_b200 import lsa

        if "call" not in s:
            s["call"] = lsa.fp8_append(lsa.LsaConfig(), s["slot"], s["latent"], s["latent_pages"], s["k"], s["key_pages"], bind=True)
        s["call"]()
        return _seen(s["latent_pages"], s["key_pages"])
    at = torch.where(s["slot"] >= 0)[0]
    slot = s["slot"][at].long()

    def put(pool, x):
        rows = pool.view(-1, LAT_ROW)
        codes, scale = _quant(x[at].float())
        rows[slot, :LAT] = codes.view(torch.uint8)
        rows[slot, LAT:LAT + 4] = scale.view(torch.uint8)

    [put(p, x) for p, x in zip(s["latent_pages"], s["latent"])]
    codes, scale = _quant(s["k"][at].float())
    pages = s["key_pages"]
    pages[:, :PAGE * KEY].view(-1, PAGE, KEY)[slot // PAGE, slot % PAGE] = codes.view(torch.uint8)
    pages.view(torch.float32)[slot // PAGE, PAGE * KEY // 4 + slot % PAGE] = scale[:, 0]
    return _seen(s["latent_pages"], s["key_pages"])


def _run_scores(s):
    if own:
        from sparse_attention_03_b200 import lsa

        if "call" not in s:
            cfg = lsa.LsaConfig(index_topk=s["topk"], index_init_tokens=s["init"], index_local_tokens=s["local"])
            s["ws"] = lsa.workspace(cfg, lsa.OP_FP8_INDEX, s["pos"].numel(), s["table"].shape[0], s["max_len"])
            s["call"] = lsa.fp8_index_scores(cfg, s["seq"], s["pos"], s["q"], s["w"], s["key_pages"], s["table"], s["max_len"], s["scores"], s["ws"], bind=True)
        s["call"]()
        return s["scores"]
    n_seq, length = s["table"].shape[0], s["max_len"]
    # every sequence's keys, and its rows side by side: one product for each sequence
    page = s["table"].clamp(min=0).long()
    codes = s["key_pages"][:, :PAGE * KEY].view(F8).view(-1, PAGE, KEY)
    keys = codes.view(torch.uint8)[page].view(F8).float() * s["key_pages"].view(torch.float32)[:, PAGE * KEY // 4:][page][..., None]
    keys = keys.view(n_seq, -1, KEY)[:, :length]
    q8, sq = _quant(s["q"].float())
    real = s["seq"] >= 0
    seq = torch.where(real, s["seq"], torch.full_like(s["seq"], n_seq)).long()  # the padding rows: a sequence of their own
    rank, most = s["rank"], s["most"]
    q = torch.zeros(n_seq + 1, most, HEADS, KEY, device=seq.device)
    q[seq, rank] = q8.float() * sq
    dots = torch.bmm(q[:n_seq].view(n_seq, most * HEADS, KEY), keys.transpose(1, 2)).clamp_(min=0)
    w = torch.zeros(n_seq + 1, most, 1, HEADS, device=seq.device)
    w[seq, rank, 0] = s["w"]
    sums = torch.matmul(w[:n_seq], dots.view(n_seq, most, HEADS, length))[:, :, 0]
    scores = sums[seq.clamp(max=n_seq - 1), rank]
    j, p = torch.arange(length, device=seq.device)[None], s["pos"][:, None]
    scores = torch.where((j < s["init"]) | (j > p - s["local"]), torch.full_like(scores, math.inf), scores)
    return torch.where((j <= p) & real[:, None], scores, torch.full_like(scores, -math.inf))


SCALE = 1.0 / math.sqrt(192.0)


def _run_mla(s):
    if own:
        from sparse_attention_03_b200 import lsa

        if "call" not in s:
            cfg = lsa.LsaConfig(index_topk=s["topk"], index_init_tokens=min(16, s["topk"] // 4), index_local_tokens=min(1024, s["topk"] // 2), cli_factor=s["n_sub"])
            s["ws"] = lsa.workspace(cfg, lsa.OP_FP8_MLA, s["pos"].numel(), s["table"].shape[0], s["max_len"])
            s["call"] = lsa.fp8_sparse_mla(cfg, s["seq"], s["pos"], s["q"], s["latent_pages"], s["table"], s["idx"], s["count"], s["max_len"], s["out"], s["lse"], s["ws"], bind=True)
        s["call"]()
        return {"out": s["out"], "lse": s["lse"]}
    real = s["seq"] >= 0
    there = (torch.arange(s["topk"], device=real.device)[None] < s["count"][:, None]) & real[:, None]
    key = s["idx"].clamp(min=0).long()
    slot = s["table"][s["seq"].clamp(min=0).long()[:, None], key // PAGE].long().clamp(min=0) * PAGE + key % PAGE

    def attend(q, pool):
        rows = pool.view(-1, LAT_ROW)
        c = rows[:, :LAT][slot].view(F8).float() * rows.view(torch.float32)[:, LAT // 4][slot][..., None]
        x = torch.matmul(q.float(), c.transpose(1, 2)) * SCALE
        x = torch.where(there[:, None], x, torch.full_like(x, -math.inf))
        top = x.amax(-1, keepdim=True).clamp(min=-1e30)
        e = torch.exp(x - top)
        total = e.sum(-1, keepdim=True)
        o = torch.matmul(e, c[..., :VALUES]) / total
        lse = (top + torch.log(total))[..., 0]
        return torch.where(real[:, None, None], o, torch.zeros_like(o)).bfloat16(), torch.where(real[:, None], lse, torch.zeros_like(lse))

    both = [attend(q, p) for q, p in zip(s["q"], s["latent_pages"])]
    return {"out": [b[0] for b in both], "lse": [b[1] for b in both]}


# ---- the definitions in 64 bits


def _round_e4m3(y):
    """fp64 values of |y| <= 448 to the nearest e4m3 value, ties to even: steps of 2^(E-3), no finer than 2^-9."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_quant(x):
    a = x.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(a / 448.0)).clamp(min=-126.0))
    s = torch.where(a > 448.0 * s, s * 2, torch.where((a <= 224.0 * s) & (s > 2.0 ** -126), s / 2, s))
    s = torch.where(a > 0, s, torch.ones_like(s))
    return _round_e4m3(x / s), s


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "append":
        keep = s["slot"] >= 0
        slot = s["slot"][keep].long()
        n = case["pages"] * PAGE
        codes, scales = [], []
        for x in s["latent"] + [s["k"]]:
            c, a = _exact_quant(x.double()[keep])
            codes.append(torch.zeros(n, c.shape[1], dtype=f64, device="cuda").index_copy_(0, slot, c))
            scales.append(torch.zeros(n, dtype=f64, device="cuda").index_copy_(0, slot, a[:, 0]))
        return {"latent": codes[:-1], "latent_scale": scales[:-1], "key": codes[-1].view(-1, PAGE * KEY), "key_scale": scales[-1].view(-1, PAGE)}
    lens, rows = _geometry(case)
    n = len(rows) + case["pad"]
    if case["op"] == "scores":
        out = torch.full((n, s["max_len"]), -math.inf, dtype=f64, device="cuda")
        q8, sq = _exact_quant(s["q"].double())
        q = q8 * sq
        for b in range(case["n_seq"]):
            pages = s["key_pages"][s["table"][b, :-(-lens[b] // PAGE)].long()]
            k = (pages[:, :PAGE * KEY].view(F8).to(f64).view(-1, PAGE, KEY) * pages.view(torch.float32)[:, PAGE * KEY // 4:, None].to(f64)).view(-1, KEY)[:lens[b]]
            mine = [i for i, r in enumerate(rows) if r[0] == b]
            for at in range(0, len(mine), 64):
                i = torch.tensor(mine[at:at + 64], device="cuda")
                d = torch.einsum("rhd,jd->rhj", q[i], k).relu()
                v = torch.einsum("rh,rhj->rj", s["w"][i].double(), d)
                j, p = torch.arange(lens[b], device="cuda")[None], s["pos"][i].long()[:, None]
                v = v.masked_fill((j < case["init"]) | (j > p - case["local"]), math.inf).masked_fill(j > p, -math.inf)
                out[i, :lens[b]] = v
        return out
    outs, lses = [], []
    for q, pool in zip(s["q"], s["latent_pages"]):
        o = torch.zeros(n, HEADS, VALUES, dtype=f64, device="cuda")
        l = torch.zeros(n, HEADS, dtype=f64, device="cuda")
        flat = pool.view(-1, LAT_ROW)
        for r0 in range(0, len(rows), 64):
            i = torch.arange(r0, min(r0 + 64, len(rows)), device="cuda")
            key = s["idx"][i].long()
            there = torch.arange(case["topk"], device="cuda")[None] < s["count"][i][:, None]
            key = torch.where(there, key, torch.zeros_like(key))
            page = torch.gather(s["table"][s["seq"][i].long()].long(), 1, key // PAGE)
            c = flat[page * PAGE + key % PAGE]
            c = c[..., :LAT].contiguous().view(F8).to(f64) * c[..., LAT:LAT + 4].contiguous().view(torch.float32).to(f64)
            x = torch.einsum("rhd,rkd->rhk", q[i].double(), c) / 192.0 ** 0.5
            x = x.masked_fill(~there[:, None], -math.inf)
            l[i] = torch.logsumexp(x, -1)
            o[i] = torch.einsum("rhk,rkd->rhd", torch.exp(x - l[i][..., None]), c[..., :VALUES])
        outs.append(o)
        lses.append(l)
    return {"out": outs, "lse": lses}
