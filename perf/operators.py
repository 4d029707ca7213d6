"""What is measured of the operators beside the focal, gather and R-SWA layers.

Four operators over the paged KV cache [pages, H_kv, page, d] (one layer each):

* ``shared`` -- decode attention of a batch whose sequences share long prefixes
  in groups: sequences start[i] .. start[i+1]-1 read the keys [0, P) through the
  block table of the group's first sequence and [P, N_b) through their own.
* ``cross``  -- attention of packed, ragged queries to an encoder's states:
  rows q_start[b] .. q_start[b+1]-1 attend to all N_b states of sequence b.
* ``weigh``  -- decode attention that adds every token's attention weight,
  summed over the query heads of its KV head, to an accumulator; the row of the
  current token is set instead of added to and gets its position.
* ``evict``  -- cuts the rows behind `protect` to `budget` rows a KV head: the
  `recent` newest positions stay, then the rows of largest weight (ties to the
  lower row). Row i of the kept ones behind the budget moves into hole i of
  those before it, K, V, weight and position together.

``run`` computes them in elementary torch operations where ``own`` is false and
through the package where it is true.
"""
import math
import random

import torch

own = False


def _case(name, op, dtype, batch, q_heads, kv_heads, head_dim, page, **kw):
    return dict(name=name, op=op, dtype=dtype, batch=batch, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, page=page, **kw)


def listed():
    return [
        # four fields read from one small image: a call as short as they come, fp32
        _case("shared_small_f32", "shared", "f32", 4, 4, 2, 64, 16, groups=1, prefix=272, tail=32),
        # eight answers sampled from one page of 64x64 image tokens
        _case("shared_page_b8", "shared", "bf16", 8, 28, 4, 128, 16, groups=1, prefix=4160, tail=512),
        # 32 questions about one dense page of 128x64 image tokens
        _case("shared_serving_b32", "shared", "bf16", 32, 28, 4, 128, 16, groups=1, prefix=8320,
              tail=256),
        # four documents of four pages each, 64 long answers in uneven groups
        _case("shared_multipage_b64", "shared", "bf16", 64, 28, 4, 128, 16, groups=4, prefix=16448,
              tail=4096),
        # three short ragged requests to a small encoder, fp32
        _case("cross_small_f32", "cross", "f32", 3, 4, 2, 64, 16, queries=5, states=300),
        # one decode token a sequence, multi-head attention to the visual tokens of a page
        _case("cross_token_b16", "cross", "bf16", 16, 10, 10, 128, 16, queries=1, states=2624),
        # chunks of a prompt, one of the sequences without any encoder states
        _case("cross_chunk_b8", "cross", "bf16", 8, 28, 4, 128, 16, queries=64, states=4160),
        # whole decoder inputs against dense pages
        _case("cross_prefill_b4", "cross", "bf16", 4, 28, 4, 128, 16, queries=1024, states=8320),
        # one sequence: prompt and image protected, up to 512 generated tokens weighed
        _case("weigh_page_b1", "weigh", "bf16", 1, 28, 4, 128, 16, protect=4160, rows=512),
        # 32 sequences that hold little but the weighed rows
        _case("weigh_text_b32", "weigh", "bf16", 32, 28, 4, 128, 16, protect=128, rows=1088),
        # the steady decode step: one token over the budget, one row goes
        _case("evict_step_b8", "evict", "bf16", 8, 28, 4, 128, 16, protect=128, rows=513, budget=512,
              recent=128, ragged=False),
        # a dense page's tokens cut to an eighth once its prompt has been read
        _case("evict_prompt_b32", "evict", "bf16", 32, 28, 4, 128, 16, protect=128, rows=8192,
              budget=1024, recent=128, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "cross", "weigh", "evict"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    hq, hkv, d = rng.choice([(28, 4, 128), (10, 10, 128), (4, 2, 64), (16, 2, 128), (15, 3, 64),
                             (7, 1, 128)])
    page = rng.choice([1, 4, 16, 16, 32, 128])
    c = dict(op=op, dtype=dtype, q_heads=hq, kv_heads=hkv, head_dim=d, page=page)
    f32 = dtype == "f32"
    if op == "shared":
        b = _log_int(rng, 1, 16 if f32 else 256 // max(hkv, 4))
        c.update(batch=b, groups=rng.randint(1, min(4, b)), prefix=_log_int(rng, 40, 2100 if f32 else 16448),
                 tail=_log_int(rng, 1, 300 if f32 else 1500))
    elif op == "cross":
        b = _log_int(rng, 1, 8)
        c.update(batch=b, queries=_log_int(rng, 1, 40 if f32 else 512), states=_log_int(rng, 1, 1500 if f32 else 8320))
    elif op == "weigh":
        b = _log_int(rng, 1, 8 if f32 else 32)
        c.update(batch=b, protect=rng.choice([0, rng.randint(1, 4200)]), rows=_log_int(rng, 1, 1100))
    else:
        b = _log_int(rng, 1, 128 // max(hkv, 4))
        rows = _log_int(rng, 2, 8192)
        budget = max(1, int(rows * rng.uniform(0.05, 1.0)))
        c.update(batch=b, protect=rng.randint(0, 300), rows=rows, budget=budget,
                 recent=rng.randint(0, budget), ragged=rng.random() < 0.5)
    return c


def _lens(n, lo, hi, salt):
    """n whole numbers of [lo, hi] that go by the case alone; the largest is hi."""
    r = random.Random("%d %d %d %s" % (n, lo, hi, salt))
    v = [r.randint(lo, hi) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _plan(c):
    """The lengths of a case: key counts of every sequence and what the operator adds to them."""
    b, op = c["batch"], c["op"]
    if op == "shared":
        r = random.Random("%d %d" % (b, c["groups"]))
        cuts = sorted(r.sample(range(1, b), c["groups"] - 1)) if c["groups"] > 1 else []
        start = [0] + cuts + [b]
        plen = _lens(c["groups"], max(1, c["prefix"] - c["prefix"] // 8), c["prefix"], "prefix")
        prefix = [p for i, p in enumerate(plen) for _ in range(start[i + 1] - start[i])]
        n = [p + t for p, t in zip(prefix, _lens(b, 1, c["tail"], "tail"))]
        return dict(start=start, prefix=prefix, n=n)
    if op == "cross":
        t = _lens(b, max(1, c["queries"] // 2), c["queries"], "queries")
        n = _lens(b, max(1, c["states"] // 2), c["states"], "states")
        if b >= 8:
            n[n.index(min(n))] = 0
        return dict(t=t, n=n)
    if op == "weigh":
        return dict(n=[c["protect"] + r for r in _lens(b, max(1, c["rows"] // 2), c["rows"], "rows")])
    rows = _lens(b, max(1, c["rows"] // 2), c["rows"], "rows") if c["ragged"] else [c["rows"]] * b
    return dict(n=[c["protect"] + r for r in rows])


def work(c):
    p = _plan(c)
    b, hq, hkv, d = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"]
    e = 2 if c["dtype"] == "bf16" else 4
    row = 2 * hkv * d * e          # K and V of one token
    n = p["n"]
    if c["op"] == "shared":
        lead = p["start"][:-1]
        keys = sum(p["prefix"][i] for i in lead) + sum(x - y for x, y in zip(n, p["prefix"]))
        return {"bytes": keys * row + 2 * b * hq * d * e, "flops": 4 * hq * d * sum(n)}
    if c["op"] == "cross":
        return {"bytes": sum(n) * row + 2 * sum(p["t"]) * hq * d * e,
                "flops": 4 * hq * d * sum(x * t for x, t in zip(n, p["t"]))}
    if c["op"] == "weigh":
        rows = sum(x - c["protect"] for x in n)
        return {"bytes": sum(n) * row + 2 * b * hq * d * e + 8 * rows * hkv, "flops": 4 * hq * d * sum(n)}
    # a kept row behind the budget moves: with weights in no order, the share of the rows that lies there
    rows = [x - c["protect"] for x in n]
    moved = sum((x - c["budget"]) * min(1.0, c["budget"] / x) for x in rows if x > c["budget"])
    return {"bytes": int(8 * sum(rows) * hkv + 2 * moved * row), "flops": sum(rows) * hkv}


def prepare(c, seed):
    p = _plan(c)
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    b, hq, hkv, d, ps, op = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"], c["page"], c["op"]
    cap = max(max(p["n"]), c.get("protect", 0) + c.get("rows", 0), 1)
    cols = -(-cap // ps)
    # pages in a shuffled order; a group's whole prefix pages are the first sequence's
    perm = torch.randperm(b * cols, generator=gen, device=dev).to(torch.int32).view(b, cols)
    table = perm.clone()
    if op == "shared":
        lead = torch.tensor([s for i, s in enumerate(p["start"][:-1])
                             for _ in range(p["start"][i + 1] - s)], device=dev)
        whole = torch.tensor([x // ps for x in p["prefix"]], device=dev)
        table = torch.where(torch.arange(cols, device=dev)[None] < whole[:, None], perm[lead], perm)
    shape = (b * cols, hkv, ps, d)
    k = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)
    v = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)
    n = torch.tensor(p["n"], dtype=torch.int32, device=dev)
    s = dict(case=c, k=k, v=v, table=table.contiguous(), n=n, seq=p["n"])
    # queries that look at nine keys of their sequence, as a decoder's heads do
    seq = torch.arange(b, device=dev)
    if op == "cross":
        seq = seq.repeat_interleave(torch.tensor(p["t"], device=dev))
        q_start = [0]
        for t in p["t"]:
            q_start.append(q_start[-1] + t)
        s.update(q_start=torch.tensor(q_start, dtype=torch.int32, device=dev), t=p["t"])
    at = (torch.rand(seq.numel(), 9, generator=gen, device=dev) * n[seq][:, None]).long()
    at = at.clamp(max=max(cap - 1, 0))
    keys = k[table[seq[:, None], at // ps].long(), :, at % ps].float().mean(1)    # [rows, H_kv, d]
    q = torch.randn(seq.numel(), hq, d, generator=gen, device=dev)
    s["q"] = (q + 3.0 * keys.repeat_interleave(hq // hkv, dim=1)).to(dt)
    s["out"] = torch.empty_like(s["q"])
    if op == "shared":
        s["start"], s["prefix"] = p["start"], torch.tensor(p["prefix"], dtype=torch.int32, device=dev)
        s["lead"] = lead
    if op in ("weigh", "evict"):
        cap_rows = c["rows"]
        s["protect"] = torch.full((b,), c["protect"], dtype=torch.int32, device=dev)
        s["seen"] = n + torch.randint(0, 1000, (b,), generator=gen, device=dev, dtype=torch.int32)
        # weights as attention leaves them: few rows hold most; positions in no order after evictions
        mass = torch.exp(2.0 * torch.randn(b, hkv, cap_rows, generator=gen, device=dev))
        rank = torch.rand(b, hkv, cap_rows, generator=gen, device=dev)
        count = (n - s["protect"])[:, None, None]
        rank = torch.where(torch.arange(cap_rows, device=dev) < count, rank, 2.0 + rank)
        order = rank.argsort(-1).argsort(-1)
        s["mass"], s["pos"] = mass, ((s["seen"] - 1)[:, None, None] - order).to(torch.int32)
    if op == "evict":
        s["now_mass"], s["now_pos"] = s["mass"].clone(), s["pos"].clone()
        s["new_len"] = torch.zeros(b, dtype=torch.int32, device=dev)
    if own:
        from dynamic_sparse_kv_gb300 import CrossAttention, DecodeAttention
        if op == "cross":
            s["plan"] = CrossAttention(k[None], v[None], s["table"], n, q_heads=hq, max_rows=sum(p["t"]))
        else:
            dec = DecodeAttention(k[None], v[None], s["table"], q_heads=hq)
            dec.set_seq_len(n)
            if op == "shared":
                dec.share_prefix(p["start"], s["prefix"])
            else:
                dec.track_weights(c["rows"], s["protect"], mass=s["mass"][None], pos=s["pos"][None],
                                  seen=s["seen"])
            s["plan"] = dec
    return s


def run(s):
    c = s["case"]
    if c["op"] == "shared":
        if own:
            s["plan"].shared_layer(0, s["q"], s["out"])
        else:
            s["out"].copy_(_plain_attend(s, s["q"][:, None], _shared_rows(s))[0][:, 0])
        return s["out"]
    if c["op"] == "cross":
        if own:
            s["plan"].attend(0, s["q"], s["q_start"], s["out"])
        else:
            _plain_cross(s)
        return s["out"]
    if c["op"] == "weigh":
        if own:
            s["plan"].weigh_layer(0, s["q"], s["out"])
        else:
            _plain_weigh(s)
        return {"out": s["out"], "mass": s["mass"], "pos": s["pos"]}
    # the weights of this step arrive, then rows go
    s["mass"].copy_(s["now_mass"])
    s["pos"].copy_(s["now_pos"])
    if own:
        s["plan"].evict_layer(0, c["budget"], c["recent"], s["new_len"])
    else:
        _plain_evict(s)
    return {"len": s["new_len"], "mass": s["mass"], "pos": s["pos"], "k": s["k"], "v": s["v"]}


# ---------------------------------------------------------------- plain forms


def _own_rows(s, count):
    """Page and slot of rows 0 .. count-1 of every sequence: [B, count] each."""
    ps = s["case"]["page"]
    r = torch.arange(count, device=s["k"].device)
    return s["table"][:, r // ps].long(), (r % ps).expand(s["table"].shape[0], -1)


def _shared_rows(s):
    ps = s["case"]["page"]
    r = torch.arange(max(s["seq"]), device=s["k"].device)
    mine, first = s["table"][:, r // ps], s["table"][s["lead"]][:, r // ps]
    return torch.where(r[None] < s["prefix"][:, None], first, mine).long(), (r % ps).expand(len(s["seq"]), -1)


def _plain_attend(s, q, rows):
    """q [B, T, H_q, d] over the rows (page, slot) [B, N] below each length: out [B, T, H_q, d], p [B, H_kv, T*g, N]."""
    page, slot = rows
    b, t, hq, d = q.shape
    hkv = s["k"].shape[1]
    g = hq // hkv
    k = s["k"][page, :, slot].float()                                   # [B, N, H_kv, d]
    v = s["v"][page, :, slot].float()
    x = q.float().view(b, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * g, d)
    w = x @ k.permute(0, 2, 3, 1) / math.sqrt(d)
    live = torch.arange(page.shape[1], device=w.device) < s["n"][:, None]   # [B, N]
    w = w.masked_fill(~live[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - top.masked_fill(top == -math.inf, 0.0))
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-38)
    o = w @ v.permute(0, 2, 1, 3)                                       # [B, H_kv, T*g, d]
    return o.view(b, hkv, t, g, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d), w


def _plain_cross(s):
    most = max(s["t"])
    at = s["q_start"][:-1, None].long() + torch.arange(most, device=s["q"].device)
    live = at < s["q_start"][1:, None]
    o = _plain_attend(s, s["q"][at.clamp(max=s["q"].shape[0] - 1)], _own_rows(s, max(max(s["seq"]), 1)))[0]
    s["out"].copy_(o[live])


def _plain_weigh(s):
    o, w = _plain_attend(s, s["q"][:, None], _own_rows(s, max(s["seq"])))
    s["out"].copy_(o[:, 0])
    w = w.sum(2)                                                        # [B, H_kv, N]
    i = torch.arange(s["mass"].shape[2], device=w.device)
    r = s["protect"][:, None] + i                                       # [B, rows]
    add = torch.gather(w, 2, r.clamp(max=w.shape[2] - 1).long()[:, None].expand(-1, w.shape[1], -1))
    cur = (r == s["n"][:, None] - 1)[:, None]
    old = (r < s["n"][:, None] - 1)[:, None]
    s["mass"].copy_(torch.where(cur, add, torch.where(old, s["mass"] + add, s["mass"])))
    s["pos"].copy_(torch.where(cur, s["seen"][:, None, None] - 1, s["pos"]))


def _plain_evict(s):
    c, ps = s["case"], s["case"]["page"]
    mass, pos = s["mass"], s["pos"]
    i = torch.arange(mass.shape[2], device=mass.device)
    count = (s["n"] - s["protect"])[:, None, None]
    keep = count.clamp(max=c["budget"])
    # best rows first: rows that exist, then recent ones, then by weight, then by row
    order = torch.sort(mass, dim=-1, descending=True, stable=True)[1]
    late = (pos >= s["seen"][:, None, None] - c["recent"]) & (i < count)
    cls = torch.where(i < count, late.to(torch.int32), -1).expand_as(mass)
    order = torch.gather(order, 2, torch.sort(torch.gather(cls, 2, order), dim=-1, descending=True, stable=True)[1])
    rank = torch.empty_like(order).scatter_(2, order, i.expand_as(order))
    kept = rank < keep
    hole, stay = (i < keep) & ~kept, (i >= keep) & kept
    dst = torch.sort((~hole).to(torch.uint8), dim=-1, stable=True)[1]
    src = torch.sort((~stay).to(torch.uint8), dim=-1, stable=True)[1]
    src = torch.where(i < hole.sum(-1, keepdim=True), src, dst)
    mass.scatter_(2, dst, torch.gather(mass, 2, src))
    pos.scatter_(2, dst, torch.gather(pos, 2, src))
    head = torch.arange(mass.shape[1], device=mass.device)[None, :, None]
    seq = torch.arange(mass.shape[0], device=mass.device)[:, None, None]
    rs, rd = src + s["protect"][:, None, None], dst + s["protect"][:, None, None]
    ps_, pd = s["table"][seq, rs // ps].long(), s["table"][seq, rd // ps].long()
    for x in (s["k"], s["v"]):
        x[pd, head, rd % ps] = x[ps_, head, rs % ps]
    s["new_len"].copy_(s["protect"] + keep[:, 0, 0])


# ---------------------------------------------------------------- from the definition, in 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "evict":
        return _exact_evict(s)
    k, v, table, n = s["k"].double(), s["v"].double(), s["table"].long().tolist(), s["seq"]
    ps, hkv, g, d = c["page"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=k.device)
    mass = s["mass"].double() if c["op"] == "weigh" else None
    first = s["q_start"].tolist() if c["op"] == "cross" else list(range(c["batch"] + 1))
    for b in range(c["batch"]):
        if n[b] == 0:
            continue
        rows = list(range(n[b]))
        if c["op"] == "shared":
            lead, cut = int(s["lead"][b]), int(s["prefix"][b])
            pages = [table[lead if r < cut else b][r // ps] for r in rows]
        else:
            pages = [table[b][r // ps] for r in rows]
        pages = torch.tensor(pages, device=k.device)
        slots = torch.tensor([r % ps for r in rows], device=k.device)
        for h in range(hkv):
            kh, vh = k[pages, h, slots], v[pages, h, slots]
            qh = s["q"][first[b]:first[b + 1], h * g:(h + 1) * g].double()      # [T, g, d]
            a = torch.softmax(torch.einsum("tgd,nd->tgn", qh, kh) * d ** -0.5, dim=-1)
            out[first[b]:first[b + 1], h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", a, vh)
            if mass is not None:
                a = a[0].sum(0)[c["protect"]:]
                mass[b, h, :len(a) - 1] += a[:-1]
                mass[b, h, len(a) - 1] = a[-1]
    if c["op"] == "weigh":
        return {"out": out, "mass": mass, "pos": None}
    return out


def _exact_evict(s):
    c, ps = s["case"], s["case"]["page"]
    k, v, table = s["k"].clone(), s["v"].clone(), s["table"].long().cpu()
    mass, pos = s["now_mass"].cpu().numpy().copy(), s["now_pos"].cpu().numpy().copy()
    length = []
    for b in range(c["batch"]):
        count = s["seq"][b] - c["protect"]
        keep = min(count, c["budget"])
        length.append(c["protect"] + keep)
        edge = int(s["seen"][b]) - c["recent"]
        for h in range(c["kv_heads"]):
            m, t = mass[b, h].tolist(), pos[b, h].tolist()
            best = sorted(range(count), key=lambda r: (t[r] < edge, -m[r], r))[:keep]
            stay = set(best)
            holes = [r for r in range(keep) if r not in stay]
            moves = [r for r in range(keep, count) if r in stay]
            if not holes:
                continue
            for x, y in zip(holes, moves):
                mass[b, h, x], pos[b, h, x] = mass[b, h, y], pos[b, h, y]
            hr, mr = torch.tensor(holes) + c["protect"], torch.tensor(moves) + c["protect"]
            hp, mp = table[b][hr // ps].to(k.device), table[b][mr // ps].to(k.device)
            hs, ms = (hr % ps).to(k.device), (mr % ps).to(k.device)
            k[hp, h, hs] = s["k"][mp, h, ms]
            v[hp, h, hs] = s["v"][mp, h, ms]
    return {"len": None, "mass": torch.from_numpy(mass).double(), "pos": None, "k": k.double(), "v": v.double()}
