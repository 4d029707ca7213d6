"""What is measured of the operators around a paged KV cache: how tokens get into
it, how its pages change hands, and attention to one that is held in 4 bits.

* ``write``  -- rotary positions with several axes for queries and keys, and the
  tokens' keys and values written to their rows of the cache: the last T_b rows of
  sequence b for its T_b tokens. A cache in 4 bits is read back as the values it
  stands for.
* ``attend4`` -- decode attention over a cache in 4 bits: every row ("full"), the
  text and a selection of image tokens ("gather"), or a prefix and the newest rows
  ("rswa").
* ``pages``  -- the pages of a pool change hands in all layers: reserved for the
  next tokens, shared by forked sequences and copied before one of them writes,
  released, and moved together.

A row in 4 bits: groups of 16 dimensions. With g the KV head's gain, y = x / g and a
the group's largest |y|, the group's scale s is a / 6 rounded to e4m3 (at most 448)
and an element is y / s rounded to e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives; ties to the even code); it stands for e2m1 * s * g.

``run`` computes them in elementary torch operations where ``own`` is false and
through the package where it is true.
"""
import math
import random

import torch

own = False

MODEL = dict(q_heads=28, kv_heads=4, head_dim=128, page=16)      # 28 query heads in groups of 7
MROPE = dict(axes="16 24 24", adjacent=False, base=1e6)          # time, height, width


def _case(name, op, **kw):
    return dict(name=name, op=op, **kw)


# A case has `batch` sequences of `low` to `rows` rows (the largest has `rows`); a writing one
# puts `low` to `tokens` tokens behind up to `before` rows.
def listed():
    return [
        # one decode token of one sequence into a bf16 cache: the shortest call of a step
        _case("write_token_b1", "write", dtype="bf16", **MODEL, **MROPE, batch=1, low=1, tokens=1, before=4400),
        # one decode token of 32 sequences into a cache in 4 bits
        _case("write_token_b32_fp4", "write", dtype="fp4", **MODEL, **MROPE, batch=32, low=1, tokens=1, before=8600),
        # three short prompts of a small fp32 model, two axes, neighbouring dimensions paired
        _case("write_small_f32", "write", dtype="f32", q_heads=4, kv_heads=2, head_dim=64, page=16, axes="16 16",
              adjacent=True, base=1e4, batch=3, low=5, tokens=272, before=36),
        # prompts of four dense pages (128 text + 128x64 image tokens)
        _case("write_prompt_b4_fp4", "write", dtype="fp4", **MODEL, **MROPE, batch=4, low=6001, tokens=8320, before=0),
        # a page's answer: 4096 image tokens, batch 1
        _case("attend4_page_b1", "attend4", kind="full", **MODEL, batch=1, low=1, rows=4401),
        # the steady gather layer of 32 sequences: text, 5 % of 128x64 image tokens, the answer so far
        _case("attend4_gather_b32", "attend4", kind="gather", **MODEL, batch=32, low=8321, rows=8576, start=128,
              image=8192, keep=410),
        # 16 sequences of a model without grouped heads, prefix 2624 and window 128
        _case("attend4_rswa_b16", "attend4", kind="rswa", q_heads=10, kv_heads=10, head_dim=128, page=16,
              batch=16, low=2700, rows=4096, prefix=2624, window=128),
        # a dense or focal layer of 32 sequences
        _case("attend4_serving_b32", "attend4", kind="full", **MODEL, batch=32, low=8321, rows=8576),
        # the next token of 32 sequences in 28 layers; some of them need a page for it
        _case("pages_step_b32", "pages", kind="step", **MODEL, layers=28, batch=32, low=480, rows=720, spare=64),
        # one read page sampled 31 times more: tables shared, the last page copied for each
        _case("pages_fork_b32", "pages", kind="fork", **MODEL, layers=28, batch=32, parents=1, low=1, rows=4407,
              spare=64),
        # half of 64 answers end: their pages go, the others' move together, 8 layers
        _case("pages_finish_b64", "pages", kind="finish", **MODEL, layers=8, batch=64, low=900, rows=1936, spare=200),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "attend4", "pages"])
    hq, hkv, d = rng.choice([(28, 4, 128), (10, 10, 128), (4, 2, 64), (16, 2, 128), (15, 3, 64), (7, 1, 128)])
    page = rng.choice([1, 4, 16, 16, 32, 128])
    c = dict(op=op, q_heads=hq, kv_heads=hkv, head_dim=d, page=page)
    if op == "write":
        half = d // 2
        axes = rng.choice([[half], [half // 2, half // 2], [half // 4, 3 * half // 8, 3 * half // 8]])
        b = _log_int(rng, 1, 32)
        tokens = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, 8000 // b))
        c.update(dtype=rng.choice(["bf16", "f32", "fp4", "fp4"]), axes=" ".join(map(str, axes)),
                 adjacent=rng.random() < 0.3, base=rng.choice([1e4, 1e6]), batch=b, low=rng.randint(1, tokens),
                 tokens=tokens, before=rng.choice([0, rng.randint(1, 3000)]))
    elif op == "attend4":
        b = _log_int(rng, 1, 128 // max(hkv, 4))
        n = _log_int(rng, 1, 8000)
        low = rng.randint(max(1, n // 2), n)
        c.update(kind=rng.choice(["full", "gather", "rswa"]), batch=b, low=low, rows=n)
        if c["kind"] == "gather":
            start = rng.randint(0, low // 4)
            image = rng.randint(0, low - 1 - start)
            c.update(start=start, image=image, keep=rng.randint(0, image))
        elif c["kind"] == "rswa":
            c.update(prefix=rng.randint(0, n), window=rng.choice([0, 1, rng.randint(1, 600)]))
    else:
        b = _log_int(rng, 2, 32)
        n = _log_int(rng, 1, 1500)
        c.update(kind=rng.choice(["step", "fork", "finish"]), layers=rng.randint(1, 4), batch=b,
                 low=rng.randint(max(1, n // 2), n), rows=n, spare=b + rng.randint(0, 300))
        if c["kind"] == "fork":
            c["parents"] = rng.randint(1, max(1, b // 2))
    return c


def _ceil(a, b):
    return -(-a // b)


def _lens(n, lo, hi, salt):
    """n whole numbers of [lo, hi] that go by the case alone; the largest is hi."""
    r = random.Random("%d %d %d %s" % (n, lo, hi, salt))
    v = [r.randint(lo, hi) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _plan(c):
    """(tokens written of every sequence or None, rows of every sequence)"""
    b = c["batch"]
    if c["op"] == "write":
        tokens = _lens(b, c["low"], c["tokens"], "tokens")
        return tokens, [t + x for t, x in zip(tokens, _lens(b, 0, c["before"], "before"))]
    if c.get("kind") == "fork":
        return None, _lens(c["parents"], c["low"], c["rows"], "rows") + [0] * (b - c["parents"])
    return None, _lens(b, c["low"], c["rows"], "rows")


def _axes(c):
    return [int(x) for x in c["axes"].split()]


def work(c):
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    if c["op"] == "write":
        t = sum(_plan(c)[0])
        e = 4 if c["dtype"] == "f32" else 2
        row = 2 * hkv * (d // 2 + d // 16) if c["dtype"] == "fp4" else 2 * hkv * d * e
        moved = t * (2 * hq * d * e + 2 * hkv * d * e + row + 4 * len(_axes(c)))
        moved += 4 * d * min(t, int(_positions(c).max()) + 1)      # cosines and sines
        if c["dtype"] == "fp4":                       # read back as fp32 values
            moved += t * (row + 2 * hkv * d * 4)
        return {"bytes": moved, "flops": 6 * t * (hq + hkv) * (d // 2)}
    if c["op"] == "attend4":
        keys = sum(len(x) for x in _sets(c))
        return {"bytes": keys * 2 * hkv * (d // 2 + d // 16) + 4 * c["batch"] * hq * d, "flops": 4 * hq * d * keys}
    p = _pages_plan(c)
    e = 2
    page = 2 * c["layers"] * hkv * c["page"] * d * e
    return {"bytes": 2 * p["moved"] * page + 8 * p["entries"] + 4 * p["pages"], "flops": p["pages"]}


# ---------------------------------------------------------------- plans that go by the case alone


def _positions(c):
    """[axes, T] positions of the written tokens: text, an image grid of 64 columns, text."""
    n_axes = len(_axes(c))
    out = []
    for t, n in zip(*_plan(c)):
        r = torch.arange(n - t, n)
        i = (r - 64).clamp(min=0)
        image = (r >= 64) & (r < 64 + 64 * 64)
        after = r - 64 - 64 * 64 + 128
        grid = [torch.full_like(r, 64), 64 + i // 64, 64 + i % 64]
        grid = grid[-n_axes:] if n_axes > 1 else grid[:1]
        out.append(torch.stack([torch.where(image, g, torch.where(r < 64, r, after)) for g in grid]))
    return torch.cat(out, 1)


def _axis_of_pair(c):
    return [a for a, n in enumerate(_axes(c)) for _ in range(n)]


def _sets(c):
    """Rows that every sequence attends to."""
    out = []
    for n in _plan(c)[1]:
        if c["kind"] == "full":
            out.append(range(n))
        elif c["kind"] == "rswa":
            p = min(c["prefix"], n)
            out.append(list(range(p)) + list(range(max(c["prefix"], n - c["window"]), n)))
        else:
            tail = c["start"] + c["image"]
            out.append(list(range(c["start"])) + [0] * c["keep"] + list(range(tail, n)))
    return out


def _pages_plan(c):
    """Pages held, and how many pages move: what the kinds do to the pool, counted."""
    ps, rows = c["page"], _plan(c)[1]
    held = [_ceil(n, ps) for n in rows]
    pages = sum(held) + c["spare"]
    r = random.Random("%d %d" % (len(rows), pages))
    if c["kind"] == "step":
        moved, entries = 0, len(rows)
    elif c["kind"] == "fork":
        kids = [i for i in range(c["parents"], len(rows))]
        moved = sum(1 for i in kids if rows[i % c["parents"]] % ps)
        entries = sum(held[i % c["parents"]] for i in kids)
    else:
        ends = sorted(r.sample(range(len(rows)), len(rows) // 2))
        left = sum(h for i, h in enumerate(held) if i not in ends)
        moved = int(left * (1 - left / pages))      # of pages in no order
        entries = sum(held)
        return dict(held=held, pages=pages, moved=moved, entries=entries, ends=ends)
    return dict(held=held, pages=pages, moved=moved, entries=entries)


# ---------------------------------------------------------------- inputs


def _type(c):
    return torch.float32 if c.get("dtype") == "f32" else torch.bfloat16


def prepare(c, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case=c, dev=dev)
    {"write": _prepare_write, "attend4": _prepare_attend4, "pages": _prepare_pages}[c["op"]](s, gen)
    return s


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _channels(gen, hkv, d):
    """Keys differ in size from channel to channel."""
    return torch.exp(0.7 * _randn(gen, hkv, d))


def _table(gen, c, spare=0):
    """Pages in a shuffled order: [B, columns] and how many pages there are."""
    b, cols = c["batch"], _ceil(max(_plan(c)[1]), c["page"])
    n = b * cols + spare
    return torch.randperm(n, generator=gen, device=gen.device)[:b * cols].to(torch.int32).view(b, cols), n


def _gain(gen, hkv):
    return 0.05 + 0.4 * torch.rand(1, hkv, generator=gen, device=gen.device)


def _prepare_write(s, gen):
    c, dev = s["case"], s["dev"]
    hq, hkv, d, ps, dt = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"], _type(c)
    tokens, rows = _plan(c)
    t = sum(tokens)
    # one projection's output: queries, keys and values side by side
    qkv = _randn(gen, t, hq + 2 * hkv, d)
    qkv[:, hq:hq + hkv] *= _channels(gen, hkv, d)
    qkv = qkv.to(dt).view(t, (hq + 2 * hkv) * d)
    s["q"] = qkv[:, :hq * d].view(t, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
    s["pos"] = _positions(c).to(device=dev, dtype=torch.int32).contiguous()
    s["table"], pages = _table(gen, c)
    s["n"] = torch.tensor(rows, dtype=torch.int32, device=dev)
    start = [0]
    for x in tokens:
        start.append(start[-1] + x)
    s["start"] = torch.tensor(start, dtype=torch.int32, device=dev)
    single = all(x == 1 for x in tokens)
    s["q_start"] = None if single else s["start"]
    s["out_q"] = torch.empty(t, hq, d, dtype=dt, device=dev)
    # where the tokens go
    seq = [b for b, x in enumerate(tokens) for _ in range(x)]
    row = [n - x + i for x, n in zip(tokens, rows) for i in range(x)]
    s["seq"], s["row"] = torch.tensor(seq, device=dev), torch.tensor(row, device=dev)
    s["positions"] = int(_positions(c).max()) + 1
    shape = (1, pages, hkv, ps, d)
    if c["dtype"] == "fp4":
        s["k_gain"], s["v_gain"] = _gain(gen, hkv), _gain(gen, hkv)
        s["back"] = [torch.empty(t, hkv, d, device=dev) for _ in range(2)]
    else:
        s["cache"] = [_randn(gen, *shape).to(dt) for _ in range(2)]
    if own:
        from dynamic_sparse_kv_gb300 import DecodeAttention, Fp4Cache, Rotary
        if c["dtype"] == "fp4":
            kc = Fp4Cache(1, pages, hkv, ps, d, device=dev, gain=s["k_gain"])
            vc = Fp4Cache(1, pages, hkv, ps, d, device=dev, gain=s["v_gain"])
        else:
            kc, vc = s["cache"]
        s["dec"] = DecodeAttention(kc, vc, s["table"], q_heads=hq)
        s["dec"].set_seq_len(s["n"])
        s["rotary"] = Rotary(d, _axes(c), positions=s["positions"], base=c["base"], adjacent=c["adjacent"], device=dev)


def _prepare_attend4(s, gen):
    c, dev = s["case"], s["dev"]
    hq, hkv, d, ps, b = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"], c["batch"]
    s["table"], pages = _table(gen, c)
    s["n"] = torch.tensor(_plan(c)[1], dtype=torch.int32, device=dev)
    k = _randn(gen, pages, hkv, ps, d) * _channels(gen, hkv, d)[:, None]
    v = _randn(gen, pages, hkv, ps, d)
    s["k_gain"], s["v_gain"] = _gain(gen, hkv), _gain(gen, hkv)
    at = (torch.rand(b, 9, generator=gen, device=dev) * s["n"][:, None]).long()
    keys = k[s["table"][torch.arange(b, device=dev)[:, None], at // ps].long(), :, at % ps].mean(1)   # [B, H_kv, d]
    s["k"] = _pack(k[None], s["k_gain"])
    s["v"] = _pack(v[None], s["v_gain"])
    del k, v
    q = _randn(gen, b, hq, d) + 2.0 * keys.repeat_interleave(hq // hkv, dim=1)
    s["q"] = q.to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    if c["kind"] == "gather":
        order = torch.rand(b, max(c["image"], 1), generator=gen, device=dev).argsort(1)[:, :c["keep"]]
        idx = (order.sort(1)[0] + c["start"]).to(torch.int32)
        s["idx"] = torch.zeros(b, max(c["keep"], 1), dtype=torch.int32, device=dev)
        s["idx"][:, :c["keep"]] = idx
        s["kept"] = torch.full((b,), c["keep"], dtype=torch.int32, device=dev)
        s["img"] = torch.tensor([[c["start"], c["image"]]] * b, dtype=torch.int32, device=dev)
    if own:
        from dynamic_sparse_kv_gb300 import DecodeAttention, Fp4Cache
        caches = []
        for x, gain in (("k", s["k_gain"]), ("v", s["v_gain"])):
            cache = Fp4Cache(1, pages, hkv, ps, d, device=dev, gain=gain)
            cache.codes.copy_(s[x][0])
            cache.scales.copy_(s[x][1])
            caches.append(cache)
        kw = dict(rswa_prefix=c["prefix"], rswa_window=c["window"]) if c["kind"] == "rswa" else {}
        if c["kind"] == "gather":
            kw = dict(img_range=s["img"], max_img=c["image"])
        s["dec"] = DecodeAttention(*caches, s["table"], q_heads=hq, **kw)
        s["dec"].set_seq_len(max(_plan(c)[1]))
        s["dec"].set_seq_len(s["n"])


def _prepare_pages(s, gen):
    c, dev = s["case"], s["dev"]
    hkv, d, ps, b = c["kv_heads"], c["head_dim"], c["page"], c["batch"]
    p = _pages_plan(c)
    cols = _ceil(max(_plan(c)[1]) + 1, ps)
    # the pool's state: table, pages held, references
    flat = torch.zeros(b * cols + b + p["pages"], dtype=torch.int32, device=dev)
    s["state"], s["begin"] = flat, torch.zeros_like(flat)

    def views(x):
        return x[:b * cols].view(b, cols), x[b * cols:b * cols + b], x[b * cols + b:]

    table, held, refs = views(s["begin"])
    order = torch.randperm(p["pages"], generator=gen, device=dev).to(torch.int32)
    table.fill_(-1)
    at = 0
    for i, h in enumerate(p["held"]):
        table[i, :h] = order[at:at + h]
        at += h
    refs[order[:at].long()] = 1
    held.copy_(torch.tensor(p["held"], dtype=torch.int32))
    s["table"], s["held"], s["refs"] = views(flat)
    flat.copy_(s["begin"])
    s["n0"] = torch.tensor(_plan(c)[1], dtype=torch.int32, device=dev)
    s["n"] = s["n0"].clone()
    shape = (c["layers"], p["pages"], hkv, ps, d)
    s["k"], s["v"] = (_randn(gen, *shape).to(torch.bfloat16) for _ in range(2))
    if c["kind"] == "fork":
        kids = list(range(c["parents"], b))
        s["src"] = torch.tensor([i % c["parents"] for i in kids], dtype=torch.int32, device=dev)
        s["dst"] = torch.tensor(kids, dtype=torch.int32, device=dev)
    if c["kind"] == "finish":
        s["ends"] = torch.tensor(p["ends"], dtype=torch.int32, device=dev)
    if own:
        from dynamic_sparse_kv_gb300 import DecodeAttention, PagePool
        s["dec"] = DecodeAttention(s["k"], s["v"], s["table"], q_heads=c["q_heads"])
        s["n"] = s["dec"].seq_len
        s["pool"] = PagePool(s["dec"], held=s["held"], refs=s["refs"])


# ---------------------------------------------------------------- one pass


def run(s):
    c = s["case"]
    if c["op"] == "write":
        return _run_write(s)
    if c["op"] == "attend4":
        if not own:
            s["out"].copy_(_plain_attend4(s))
        elif c["kind"] == "full":
            s["dec"].dense_step(s["q"][None], s["out"][None])
        elif c["kind"] == "rswa":
            s["dec"].rswa_step(s["q"][None], s["out"][None])
        else:
            from dynamic_sparse_kv_gb300 import fastocr_sparse_attend
            fastocr_sparse_attend(s["dec"].handle, s["q"], s["dec"].kv[0], s["img"], s["idx"], s["idx"].shape[1],
                                  s["kept"], s["out"])
        return s["out"]
    # the state that the step finds
    s["state"].copy_(s["begin"])
    s["n"].copy_(s["n0"])
    if own:
        if c["kind"] == "fork":
            s["pool"].fork(s["src"], s["dst"])
        if c["kind"] == "finish":
            s["pool"].release(s["ends"])
            s["pool"].compact()
        else:
            s["pool"].reserve(extra=1)
    else:
        if c["kind"] == "fork":
            _plain_fork(s)
        if c["kind"] == "finish":
            _plain_release(s)
            _plain_compact(s)
        else:
            _plain_reserve(s)
    return {x: s[x] for x in ("table", "held", "refs", "n", "k", "v")}


def _run_write(s):
    c = s["case"]
    if own:
        s["dec"].write_layer(0, s["k"], s["v"], q=s["q"], out_q=s["out_q"], rotary=s["rotary"], pos=s["pos"],
                             q_start=s["q_start"])
        if c["dtype"] == "fp4":
            s["dec"].read_layer(0, s["start"], *s["back"])
            return {"q": s["out_q"], "k": s["back"][0], "v": s["back"][1]}
        return {"q": s["out_q"], "k": s["cache"][0], "v": s["cache"][1]}
    cos, sin = _plain_angles(s)
    s["out_q"].copy_(_plain_rotate(c, s["q"].float(), cos, sin))
    k, v = _plain_rotate(c, s["k"].float(), cos, sin), s["v"].float()
    if c["dtype"] == "fp4":
        for x, y, gain in ((s["back"][0], k, s["k_gain"]), (s["back"][1], v, s["v_gain"])):
            x.copy_(_unpack(*_pack(y[None, None].transpose(2, 3), gain), gain)[0, 0].transpose(0, 1))
        return {"q": s["out_q"], "k": s["back"][0], "v": s["back"][1]}
    page = s["table"][s["seq"], s["row"] // c["page"]].long()
    for cache, y in zip(s["cache"], (k, v)):
        cache[0, page, :, s["row"] % c["page"]] = y.to(cache.dtype)
    return {"q": s["out_q"], "k": s["cache"][0], "v": s["cache"][1]}


# ---------------------------------------------------------------- plain forms


def _plain_angles(s):
    """cos, sin of every token and pair [T, d/2], from angles in 64 bits."""
    c = s["case"]
    half = c["head_dim"] // 2
    freq = c["base"] ** (-torch.arange(half, dtype=torch.float64, device=s["dev"]) / half)
    axis = torch.tensor(_axis_of_pair(c), device=s["dev"])
    angle = s["pos"][axis].double().T * freq
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _plain_rotate(c, x, cos, sin):
    half = c["head_dim"] // 2
    if c["adjacent"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _pack(x, gain):
    """x [L, pages, H, rows, d] fp32 -> (codes [..., d/2] uint8, low nibble first; scales [..., d/16] e4m3)."""
    y = (x / gain[:, None, :, None, None]).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    z = y / s.float()
    z = torch.where(s.float() == 0, 0.0, z)
    a = z.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for edge, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= edge) if up else (a > edge)
    code += (torch.signbit(z) & (code > 0)).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s[..., 0]


def _unpack(codes, scales, gain):
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    y = torch.stack([level[(codes & 15).long()], level[(codes >> 4).long()]], dim=-1).flatten(-2)
    y = y.unflatten(-1, (-1, 16)) * scales.float()[..., None]
    return y.flatten(-2) * gain[:, None, :, None, None]


def _plain_attend4(s):
    c = s["case"]
    hq, hkv, d, ps = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    b, most = c["batch"], c["rows"]
    r = torch.arange(most, device=s["dev"])[None]
    n = s["n"][:, None]
    live = r < n
    if c["kind"] == "rswa":
        live &= (r < c["prefix"]) | (r >= n - c["window"])
    elif c["kind"] == "gather":
        live &= (r < c["start"]) | (r >= c["start"] + c["image"])
        if c["keep"]:
            live = live.scatter(1, s["idx"].long(), True)
    page, slot = s["table"][:, r[0] // ps].long(), (r[0] % ps).expand(b, -1)
    out = torch.empty(b, hkv, hq // hkv, d, device=s["dev"])
    for h in range(hkv):      # a KV head at a time: the values take eight times the room
        k, v = (_unpack(x[0][:, page, h, slot][:, :, None], x[1][:, page, h, slot][:, :, None], gain[:, h:h + 1])[0]
                for x, gain in ((s["k"], s["k_gain"]), (s["v"], s["v_gain"])))
        k, v = k[:, 0], v[:, 0]                                         # [B, N, d]
        q = s["q"].float().view(b, hkv, hq // hkv, d)[:, h]
        w = q @ k.transpose(1, 2) / math.sqrt(d)
        w = w.masked_fill(~live[:, None], -math.inf)
        top = w.amax(-1, keepdim=True)
        w = torch.exp(w - top.masked_fill(top == -math.inf, 0.0))
        out[:, h] = (w / w.sum(-1, keepdim=True).clamp(min=1e-38)) @ v
    return out.view(b, hq, d)


def _held_mask(s):
    return torch.arange(s["table"].shape[1], device=s["dev"])[None] < s["held"][:, None]


def _count(pages, mask, size):
    """How often each page occurs under the mask."""
    at = torch.where(mask, pages, size).flatten().long()
    return torch.zeros(size + 1, dtype=torch.int32, device=pages.device).index_add_(
        0, at, torch.ones_like(at, dtype=torch.int32))[:size]


def _plain_fork(s):
    table, held, refs, n = s["table"], s["held"], s["refs"], s["n"]
    src, dst = s["src"].long(), s["dst"].long()
    refs -= _count(table[dst], _held_mask(s)[dst], refs.numel())
    take = -(-n[src] // s["case"]["page"])
    mask = torch.arange(table.shape[1], device=s["dev"])[None] < take[:, None]
    refs += _count(table[src], mask, refs.numel())
    table[dst] = torch.where(mask, table[src], -1)
    held[dst] = take.to(torch.int32)
    n[dst] = n[src]


def _plain_release(s):
    table, held, refs, n = s["table"], s["held"], s["refs"], s["n"]
    at = s["ends"].long()
    refs -= _count(table[at], _held_mask(s)[at], refs.numel())
    table[at] = -1
    held[at] = 0
    n[at] = 0


def _plain_reserve(s):
    """Pages for one more row of every sequence. A page in two tables is copied first, but for
    the first sequence that wants it where nobody else keeps it."""
    table, held, refs, n, ps = s["table"], s["held"], s["refs"], s["n"], s["case"]["page"]
    size = refs.numel()
    col = torch.arange(table.shape[1], device=s["dev"])[None]
    need = -(-(n + 1) // ps)
    first = n // ps
    mine = (col < need[:, None]) & ((col >= first[:, None]) | (col >= held[:, None]))
    have = _held_mask(s) & mine
    old = table.clamp(min=0).long()
    shared = have & (refs[old] > 1)
    wanted = _count(table, have, size)
    # the first entry of each page in order of sequence and column
    place = torch.arange(table.numel(), device=s["dev"]).view_as(table)
    lead = torch.full((size + 1,), table.numel(), device=s["dev"])
    lead.scatter_reduce_(0, torch.where(shared, old, size).flatten(), place.flatten(), "amin")
    keeps = shared & (wanted[old] == refs[old]) & (lead[old] == place)
    fresh = (mine & ~have) | (shared & ~keeps)
    rank = fresh.flatten().cumsum(0).view_as(table) - 1
    free = torch.sort((refs > 0).to(torch.uint8), stable=True)[1]       # free pages first, in order
    new = free[rank.clamp(0, size - 1)]
    # one page a sequence may hold rows and be replaced; where none is, a page in use stands for itself
    at = (n // ps).long().clamp(max=table.shape[1] - 1)[:, None]
    copied = ((fresh & have).gather(1, at) & (n % ps != 0)[:, None])[:, 0]
    from_ = torch.where(copied, old.gather(1, at)[:, 0], refs.argmax())
    to = torch.where(copied, new.gather(1, at)[:, 0], refs.argmax())
    for x in (s["k"], s["v"]):
        x[:, to] = x[:, from_]
    refs -= _count(table, fresh & have, size)
    refs += _count(new.to(torch.int32), fresh, size)
    table.copy_(torch.where(fresh, new.to(torch.int32), table))
    held.copy_(torch.maximum(held, need.to(torch.int32)))


def _plain_compact(s):
    """Used pages behind the first `used` move into the free ones before, in order."""
    table, refs = s["table"], s["refs"]
    size = refs.numel()
    page = torch.arange(size, device=s["dev"])
    used = refs > 0
    border = used.sum()
    hole, late = ~used & (page < border), used & (page >= border)
    holes = torch.sort((~hole).to(torch.uint8), stable=True)[1]
    to = torch.where(late, holes[(late.cumsum(0) - 1).clamp(min=0)], page)
    late_pages = torch.sort((~late).to(torch.uint8), stable=True)[1]
    source = torch.where(hole, late_pages[(hole.cumsum(0) - 1).clamp(min=0)], page)
    for x in (s["k"], s["v"]):
        for layer in x:
            layer.copy_(layer[source])
    refs.copy_(torch.where(page < border, refs[source], 0))
    table.copy_(torch.where(_held_mask(s), to[table.clamp(min=0).long()].to(torch.int32), table))


# ---------------------------------------------------------------- from the definition, in 64 bits


def exact(c, seed):
    if c["op"] == "pages":
        return _exact_pages(prepare(c, seed))
    s = prepare(c, seed)
    return _exact_write(s) if c["op"] == "write" else _exact_attend4(s)


def _exact_write(s):
    c = s["case"]
    d, hkv, ps = c["head_dim"], c["kv_heads"], c["page"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    pos = s["pos"].double()
    axis = _axis_of_pair(c)
    for i in range(d // 2):
        i0, i1 = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + d // 2)
        # the table that a program keeps is in 32 bits
        turn = pos[axis[i]] * c["base"] ** (-2.0 * i / d)
        co, si = torch.cos(turn).float().double()[:, None], torch.sin(turn).float().double()[:, None]
        for x in (q, k):
            x0, x1 = x[..., i0].clone(), x[..., i1].clone()
            x[..., i0] = x0 * co - x1 * si
            x[..., i1] = x1 * co + x0 * si
    if c["dtype"] == "fp4":       # what is held in 4 bits is a choice between neighbours, not a number in 64 bits
        return {"q": q, "k": None, "v": None}
    out = [x.double() for x in s["cache"]]
    table = s["table"].tolist()
    where = [(table[b][r // ps], r % ps) for b, r in zip(s["seq"].tolist(), s["row"].tolist())]
    page, slot = (torch.tensor(x, device=q.device) for x in zip(*where))
    for h in range(hkv):
        out[0][0][page, h, slot] = k[:, h]
        out[1][0][page, h, slot] = v[:, h]
    return {"q": q, "k": out[0], "v": out[1]}


def _exact_values(codes, scales, gain):
    """Rows of one KV head: codes [n, d/2], scales [n, d/16]."""
    level = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    level = torch.tensor(level + [-x for x in level], dtype=torch.float64, device=codes.device)
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    out[:, 0::2] = level[(codes % 16).int()]
    out[:, 1::2] = level[torch.div(codes, 16, rounding_mode="floor").int()]
    for g in range(scales.shape[1]):
        out[:, 16 * g:16 * g + 16] *= scales[:, g:g + 1].to(torch.float64)
    return out * float(gain)


def _exact_attend4(s):
    c = s["case"]
    hq, hkv, d, ps = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["dev"])
    table = s["table"].long().cpu()
    kept = s["idx"].cpu() if c["kind"] == "gather" else None
    for b, rows in enumerate(_sets(c)):
        rows = list(rows)
        if kept is not None:
            rows[c["start"]:c["start"] + c["keep"]] = kept[b, :c["keep"]].tolist()
        if not rows:
            continue
        rows = torch.tensor(rows)
        page, slot = table[b][rows // ps].to(s["dev"]), (rows % ps).to(s["dev"])
        for h in range(hkv):
            k, v = (_exact_values(x[0][0][page, h, slot], x[1][0][page, h, slot], gain[0, h])
                    for x, gain in ((s["k"], s["k_gain"]), (s["v"], s["v_gain"])))
            q = s["q"][b, h * g:(h + 1) * g].double()
            out[b, h * g:(h + 1) * g] = torch.softmax(q @ k.T * d ** -0.5, dim=-1) @ v
    return out


def _exact_pages(s):
    c, ps = s["case"], s["case"]["page"]
    b = c["batch"]
    table = [[x for x in row if x >= 0] for row in s["table"].tolist()]
    cols, size = s["table"].shape[1], s["refs"].numel()
    n = _plan(c)[1]
    moves = []

    def free():
        taken = {x for row in table for x in row}
        return [x for x in range(size) if x not in taken]

    if c["kind"] == "fork":
        for i in range(c["parents"], b):
            table[i], n[i] = list(table[i % c["parents"]])[:_ceil(n[i % c["parents"]], ps)], n[i % c["parents"]]
    if c["kind"] == "finish":
        for i in s["ends"].tolist():
            table[i], n[i] = [], 0
        used = size - len(free())
        holes = [x for x in free() if x < used]
        late = sorted({x for row in table for x in row if x >= used})
        moves = list(zip(late, holes))
        to = dict(moves)
        table = [[to.get(x, x) for x in row] for row in table]
    else:
        start, pool = [list(row) for row in table], free()
        writers = {}
        for i in range(b):
            col = n[i] // ps
            if col < len(start[i]):
                writers.setdefault(start[i][col], []).append(i)
        for i in range(b):
            col = n[i] // ps
            if col >= len(start[i]):
                table[i].append(pool.pop(0))
                continue
            page = start[i][col]
            holders = sum(row.count(page) for row in start)
            if holders > 1 and not (holders == len(writers[page]) and writers[page][0] == i):
                table[i][col] = pool.pop(0)
                if n[i] % ps:
                    moves.append((page, table[i][col]))
    refs = [0] * size
    for row in table:
        for x in row:
            refs[x] += 1
    k, v = s["k"].double(), s["v"].double()
    if moves:
        src, dst = (torch.tensor(x, device=k.device) for x in zip(*moves))
        k[:, dst], v[:, dst] = s["k"][:, src].double(), s["v"][:, src].double()
    return {"table": torch.tensor([row + [-1] * (cols - len(row)) for row in table]),
            "held": torch.tensor([len(row) for row in table]), "refs": torch.tensor(refs),
            "n": torch.tensor(n), "k": k, "v": v}
