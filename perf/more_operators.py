"""Cases and plain forms of the management of a paged KV cache's pages and of sparse attention over pages that a cheap score
chooses. They work on the cache of `operators.py`: pages of [kv head, slot, head_dim] rows in bf16, e4m3 or int8.

The pages of a pool are counted: refs[p] is how many requests hold page p, 0 a free page. Request r holds the first
ceil(lens[r] / page size) entries of its row of the page table.

  resize   lens become want: pages behind the new length are let go, and requests that grow get the lowest free pages, in
           their order; one that grows into a partly filled page that others hold gets a copy of it
  fork     row r of the table becomes a copy of row parents[r], which shares its pages
  compact  pages move from the top of the pool to the free ones below, and the tables follow
  copy     the contents of the pages that resize and compact name

  bounds   for each page that has become full and kv head the least and the greatest key of every channel, int8
  select   for each query row and kv head the pages whose bounds allow the greatest scores
  sparse   attention of a query row over its chosen pages, the rest of the prefix behind the last full page, and its tree"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "e4m3": E4M3, "i8": torch.int8}
TOP = {"e4m3": 448.0, "i8": 127.0}


def listed():
    # resize and copy are timed in every life of fork and compact too, as a server calls them
    return [
        # a step of beam search: 4 users with 8 beams each, whose tables are reordered, grow by a token and part at their last page
        dict(name="fork_beams", op="fork", groups=4, width=8, prefix=2000, tail=70, grow=1, hkv=8, dim=128, page=16, type="bf16", layers=1, life="beams"),
        # 8 samples of each of 64 prompts are let go, forked anew and grow by a drafted block; two layers share the tables
        dict(name="fork_samples", op="fork", groups=64, width=8, prefix=8192, tail=0, grow=16, hkv=8, dim=128, page=16, type="e4m3", layers=2, life="samples"),
        # a server of 512 requests whose halves come and go, on a pool of half a million pages
        dict(name="resize_churn", op="resize", n_req=512, length=16384, page=16),
        # a few requests end, the pool is packed, others begin
        dict(name="compact_small", op="compact", n_req=8, length=500, hkv=4, dim=64, page=20, type="bf16"),
        # the same on a full server, where the copies are what takes the time
        dict(name="compact_large", op="compact", n_req=128, length=8192, hkv=8, dim=128, page=32, type="e4m3"),
        # the pages that a step of 256 requests has filled
        dict(name="bounds_step", op="bounds", n_req=256, length=3000, more=16, hkv=8, dim=128, page=16, type="bf16"),
        # whole prompts
        dict(name="bounds_prompts", op="bounds", n_req=64, length=0, more=8192, hkv=8, dim=128, page=64, type="e4m3"),
        # one token over a long context: 8192 pages, of which it takes 128
        dict(name="select_1", op="select", n_req=1, nodes=1, prefix=131072, hq=32, hkv=8, dim=128, page=16, take=128),
        # drafted blocks of 16 of 32 requests, each node with its own choice
        dict(name="select_block16", op="select", n_req=32, nodes=16, prefix=32768, hq=32, hkv=8, dim=128, page=16, take=128),
        # one token of one request over its 32 chosen pages of 64, where latency is all
        dict(name="sparse_1", op="sparse", n_req=1, nodes=1, prefix=131072, hq=32, hkv=8, dim=128, page=64, take=32, type="bf16", mask="chain"),
        # plain decoding of 128 requests over an e4m3 cache, 8 query heads to a kv head
        dict(name="sparse_r128", op="sparse", n_req=128, nodes=1, prefix=32768, hq=64, hkv=8, dim=128, page=32, take=64, type="e4m3", mask="chain"),
        # the verify pass of 32 drafted trees of 16, whose nodes choose much the same pages
        dict(name="sparse_tree16", op="sparse", n_req=32, nodes=16, prefix=16384, hq=32, hkv=8, dim=128, page=16, take=128, type="bf16", mask="tree"),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["fork", "resize", "compact", "bounds", "select", "select", "sparse", "sparse", "sparse"])
    page = rng.choice([8, 16, 16, 20, 32, 64, 100, 128])
    c = dict(op=op, page=page)
    if op == "resize":
        return c | dict(n_req=_spread(rng, 1, 512), length=_spread(rng, 1, 16384))
    c |= dict(hkv=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 128, 256]), type=rng.choice(["bf16", "e4m3", "i8"]))
    if op == "fork":
        c |= dict(groups=_spread(rng, 1, 64), width=rng.randint(1, 8), prefix=_spread(rng, 1, 8192), tail=rng.randint(1, 100), grow=_spread(rng, 1, 40), layers=rng.randint(1, 2))
        c["life"] = rng.choice(["beams", "samples"])
        most, at, shrink = 2e9, "prefix", lambda: _pool_bytes(c, c["groups"] * (c["prefix"] + page + c["width"] * (c["tail"] + c["grow"] + 2 * page))) * c["layers"]
    elif op == "compact":
        c |= dict(n_req=_spread(rng, 2, 128), length=_spread(rng, 1, 8192))
        most, at, shrink = 1.0e9, "length", lambda: _pool_bytes(c, c["n_req"] * (c["length"] + page))
    elif op == "bounds":
        c |= dict(n_req=_spread(rng, 1, 256), length=rng.choice([0, 1, 50, 1000]), more=_spread(rng, 1, 8192))
        most, at, shrink = 0.28e9, "more", lambda: _pool_bytes(c, c["n_req"] * (c["length"] + c["more"] + page)) / 2
    else:
        c |= dict(n_req=_spread(rng, 1, 128), nodes=rng.choice([1, 1, 2, 5, 10, 16, 33]), prefix=_spread(rng, 1, 131072), take=_spread(rng, 2, 256))
        c["hq"] = c["hkv"] * rng.choice([1, 2, 3, 4, 5, 7, 8])
        if op == "select":
            del c["type"]
            c["prefix"] = max(c["prefix"], page * (c["take"] + 8))  # so that there is a choice
            most, at, shrink = 2.1e9, "prefix", lambda: c["n_req"] * c["nodes"] * c["hq"] * (c["prefix"] / page) * c["dim"]
        else:
            c["mask"] = rng.choice(["chain", "tree", "full"])
            c["n_req"] = max(1, min(c["n_req"], int(4.3e9 / (c["nodes"] * c["hkv"] * (min(c["take"] * page, c["prefix"]) + page + c["nodes"]) * c["dim"] * 4))))
            most, at, shrink = 4.3e9, "prefix", lambda: _pool_bytes(c, c["n_req"] * (c["prefix"] + c["nodes"] + page))
    while shrink() > most or work(c)["bytes"] > 1.0e9:
        at = "take" if op == "select" and c["prefix"] < 2 * page * (c["take"] + 8) and c["n_req"] == 1 else "n_req" if op == "select" and c["n_req"] > 1 else at
        c[at if c[at] > page or "n_req" not in c else "n_req"] //= 2
    return c


def _pool_bytes(c, tokens):
    """Bytes of K and V rows."""
    return tokens * 2 * c["hkv"] * (c["dim"] * 2 if c["type"] == "bf16" else c["dim"] + 1)


def _lengths(most, n, least=1):
    """n whole numbers up to `most`, the first of them `most`, spread evenly over least .. most: a batch's lengths."""
    return np.array([most if r == 0 else least + int((most - least) * ((r * 0.6180339887) % 1.0)) for r in range(n)], dtype=np.int64)


def _pages(tokens, page):
    return -(-tokens // page)


def _halves(c):
    """Lengths of the requests in the two states that a server goes to and fro between: either half is gone in one of them."""
    n = c["n_req"]
    lens = _lengths(c["length"], n)
    first = np.arange(n) % 2 == 0
    return np.where(first, lens, 0), np.where(first, 0, lens)


def _batch(c):
    """(start, rows) of each request of a step with drafted nodes. One has no prefix and one no rows, where there are many."""
    n = c["n_req"]
    start, rows = _lengths(c["prefix"], n, c["prefix"] // 2), np.full(n, c["nodes"])
    if n >= 16:
        start[n // 2], rows[n // 3] = 0, 0
    return start, rows


def _ends(c):
    """(start, end) of the positions that a step has filled."""
    n = c["n_req"]
    start = _lengths(c["length"], n, c["length"] // 2) if c["length"] else np.zeros(n, dtype=np.int64)
    return start, start + _lengths(c["more"], n, 1)


def work(case):
    c, page = case, case["page"]
    if c["op"] == "resize":
        a, b = _halves(c)
        pages = int(_pages(a, page).sum()) + int(_pages(b, page).sum())
        return {"bytes": 4 * (_churn_pages(c) + pages * 3 + 4 * c["n_req"]), "flops": 0}
    if c["op"] == "fork":
        lens, rows = _fork_lens(c), c["groups"] * (c["width"] + (c["life"] == "samples"))
        shared = int(_pages(lens, page).sum()) * c["width"]
        return {"bytes": 4 * (3 * shared + 6 * rows) + 2 * _pool_bytes(c, page) * c["layers"] * int((lens % page != 0).sum()) * (c["width"] // 2 if c["life"] == "beams" else c["width"]), "flops": 0}
    if c["op"] == "compact":
        a, b = (int(_pages(x, page).sum()) for x in _halves(c))
        return {"bytes": 4 * (3 * (a + b)) + 2 * _pool_bytes(c, page) * min(a, b), "flops": 0}
    if c["op"] == "bounds":
        start, end = _ends(c)
        full = int((end // page - start // page).sum())
        return {"bytes": full * (_pool_bytes(c, page) // 2 + c["hkv"] * (2 * c["dim"] + 1) + 4), "flops": 0}
    start, rows = _batch(c)
    n, hq, hkv, dim = int(rows.sum()), c["hq"], c["hkv"], c["dim"]
    blocks = start // page
    if c["op"] == "select":
        seen = int((blocks * (rows > 0)).sum())
        return {"bytes": seen * (hkv * (2 * dim + 1) + 4) + n * (hq * dim * 2 + hkv * c["take"] * 4), "flops": int((blocks * rows).sum()) * 4 * hq * dim}
    taken = np.minimum(blocks, c["take"]) * page + start % page
    # of a request's rows each page at least once
    seen = int(((taken + rows) * (rows > 0)).sum())
    flops = int((taken * rows + rows * (rows + 1) // 2).sum()) * 4 * hq * dim
    return {"bytes": int(_pool_bytes(c, seen)) + n * (2 * hq * dim * 2 + hkv * c["take"] * 4), "flops": flops}


# --- inputs ---


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _ints(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _random_codes(gen, shape, kind):
    """Rows of a cache as they would be after a write, and their scales."""
    x = _normal(gen, *shape)
    x[..., :2] *= 6
    return _quantise(x, kind)


def _quantise(x, kind):
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    top_m, top_e = math.frexp(TOP[kind])
    e = torch.where(amax > 0, e - top_e + (m > top_m), -100).clamp(min=-100)
    y = torch.ldexp(x, -e[..., None])
    return (y.to(E4M3) if kind == "e4m3" else y.round().to(torch.int8)), (e + 127).to(torch.uint8)


def _cache(gen, c, n_pages):
    """A layer's cache full of rows, made 2^14 rows at a time."""
    shape = (n_pages, c["hkv"], c["page"])
    out = dict(k_scale=None, v_scale=None)
    for name in "kv":
        out[name] = torch.empty(shape + (c["dim"],), dtype=TYPES[c["type"]], device="cuda")
        if c["type"] != "bf16":
            out[name + "_scale"] = torch.empty(shape, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (c["hkv"] * c["page"] * c["dim"]))
        for at in range(0, n_pages, step):
            codes, scale = _random_codes(gen, (min(step, n_pages - at),) + shape[1:] + (c["dim"],), c["type"])
            out[name][at : at + step] = codes
            if scale is not None:
                out[name + "_scale"][at : at + step] = scale
    return out


def _fork_lens(c):
    """Positions that each group's prompt, and each beam, has."""
    return _lengths(c["prefix"], c["groups"], c["prefix"] // 2 + 1) + (c["tail"] if c["life"] == "beams" else 0)


def _churn_pages(c):
    a, b = (int(_pages(x, c["page"]).sum()) for x in _halves(c))
    return a + b + 7 + _kept(c)


def _kept(c):
    """Pages that belong to no request: a cache of prompts holds them."""
    return int(_pages(c["length"], c["page"])) + 5


def _random_table(rnd, lens, page, width, n_pages):
    """Tables whose requests hold pages of their own from all over the pool."""
    need = _pages(lens, page)
    table = np.full((len(lens), width), -1, dtype=np.int64)
    table[np.arange(width)[None] < need[:, None]] = rnd.permutation(n_pages)[: int(need.sum())]
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = np.random.RandomState(seed % (1 << 31))
    make = {"fork": _prepare_fork, "resize": _prepare_halves, "compact": _prepare_halves, "bounds": _prepare_bounds, "select": _prepare_select, "sparse": _prepare_sparse}
    s = make[case["op"]](case, gen, rnd)
    s["case"], s["turn"] = case, 0
    return s


def _books(s, refs, table, lens, n_copies):
    s |= dict(refs=_ints(refs), table=_ints(table), lens=_ints(lens), copies=torch.zeros((max(1, n_copies), 2), dtype=torch.int32, device="cuda"), counts=torch.zeros(2, dtype=torch.int32, device="cuda"))
    return s


def _prepare_fork(c, gen, rnd):
    page, groups, w = c["page"], c["groups"], c["width"]
    lens = _fork_lens(c)
    beams = c["life"] == "beams"
    per = w if beams else w + 1
    shared = lens // page if not beams else (lens - c["tail"]) // page  # whole pages of the prompt
    need = _pages(lens, page)
    ways = 8 if beams else 1
    width = int(_pages(lens.max() + c["grow"] * ways, page)) + 1
    spare = groups * per * (int(_pages(c["grow"] * ways, page)) + 2)
    n_pages = int((shared + (need - shared) * (per if beams else 1)).sum()) + spare
    order = rnd.permutation(n_pages)
    table, refs, at = np.full((groups * per, width), -1, dtype=np.int64), np.zeros(n_pages, dtype=np.int64), 0
    for g in range(groups):
        prompt = order[at : at + shared[g]]
        at += shared[g]
        for i in range(per if beams else 1):
            mine = order[at : at + need[g] - shared[g]]
            at += need[g] - shared[g]
            table[g * per + i, : need[g]] = np.concatenate([prompt, mine])
            refs[table[g * per + i, : need[g]]] += 1
    s = {}
    every = np.repeat(lens, per)
    if beams:
        parents = np.arange(groups * per) // per * per + rnd.randint(0, per, groups * per)
        s["wants"] = [_ints(every + c["grow"] * (i + 1)) for i in range(ways)]
    else:
        child = np.arange(groups * per) % per != 0
        parents = np.arange(groups * per) // per * per
        s["wants"] = [_ints(np.where(child, 0, every)), _ints(every + child * c["grow"])]
        every = np.where(child, 0, every)
    s["parents"] = _ints(parents)
    s["layers"] = [_cache(gen, c, n_pages) for _ in range(c["layers"])]
    return _books(s, refs, table, every, groups * per)


def _prepare_halves(c, gen, rnd):
    page = c["page"]
    a, b = _halves(c)
    n_pages, width = _churn_pages(c), int(_pages(c["length"], page)) + 1
    lens = b if c["op"] == "resize" else a + b
    table = _random_table(rnd, lens, page, width, n_pages)
    refs = np.bincount(table[table >= 0], minlength=n_pages)
    refs[rnd.choice(np.nonzero(refs == 0)[0], size=_kept(c), replace=False)] = 1
    s = dict(wants=[_ints(a), _ints(b), _ints(a + b)])
    if c["op"] == "compact":
        s["layers"] = [_cache(gen, c, n_pages)]
        s["map"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    return _books(s, refs, table, lens, max(c["n_req"], n_pages // 2))


def _prepare_bounds(c, gen, rnd):
    start, end = _ends(c)
    width, n_pages = int(_pages(end.max(), c["page"])), int(_pages(end, c["page"]).sum()) + 3
    s = _cache(gen, c, n_pages)
    s |= dict(table=_ints(_random_table(rnd, end, c["page"], width, n_pages)), start=_ints(start), end=_ints(end))
    s["low_high"] = torch.zeros((n_pages, c["hkv"], 2, c["dim"]), dtype=torch.int8, device="cuda")
    s["unit"] = torch.zeros((n_pages, c["hkv"]), dtype=torch.uint8, device="cuda")
    return s


def _prepare_batch(c, rnd):
    start, rows = _batch(c)
    total = start + rows
    width, n_pages = int(max(1, _pages(total.max(), c["page"]))), int(_pages(total, c["page"]).sum()) + 3
    s = dict(table=_ints(_random_table(rnd, total, c["page"], width, n_pages)), start=_ints(start), offsets=_ints(np.concatenate([[0], np.cumsum(rows)])))
    s["n_rows"] = int(rows.sum()) + 3  # a few rows of padding behind the last request's
    return s, n_pages


def _queries(gen, c, n_rows):
    packed = _normal(gen, n_rows, c["hq"] + 2 * c["hkv"], c["dim"])
    packed[..., :2] *= 3
    return packed.to(torch.bfloat16)[:, : c["hq"]]


def _prepare_select(c, gen, rnd):
    s, n_pages = _prepare_batch(c, rnd)
    # a page's keys lie around a point of their own, a few channels far out
    shape = (n_pages, c["hkv"], c["dim"])
    mid, half = _normal(gen, *shape) * 16, _normal(gen, *shape).abs() * 9 + 6
    mid[..., :2] *= 3
    s["low_high"] = torch.stack([(mid - half).floor(), (mid + half).ceil()], dim=2).clamp(-127, 127).to(torch.int8)
    s["unit"] = torch.randint(121, 124, shape[:2], generator=gen, device="cuda").to(torch.uint8)
    s["q"] = _queries(gen, c, s["n_rows"])
    s["chosen"] = torch.full((s["n_rows"], c["hkv"], c["take"]), -1, dtype=torch.int32, device="cuda")
    return s


def _prepare_sparse(c, gen, rnd):
    s, n_pages = _prepare_batch(c, rnd)
    start, rows = _batch(c)
    s |= _cache(gen, c, n_pages)
    n_rows, take = s["n_rows"], c["take"]
    s["q"] = _queries(gen, c, n_rows)
    s["out"] = torch.zeros((n_rows, c["hq"], c["dim"]), dtype=torch.bfloat16, device="cuda")
    s["scale"] = c["dim"] ** -0.5
    # the pages that the rows have chosen: a request's rows and heads agree on most
    req = np.concatenate([np.repeat(np.arange(c["n_req"]), rows), np.zeros(n_rows - rows.sum(), dtype=np.int64)])
    blocks = torch.from_numpy(start // c["page"]).cuda()[torch.from_numpy(req).cuda()]
    most = max(1, int(start.max()) // c["page"])
    liked = torch.rand(c["n_req"], c["hkv"], most, generator=gen, device="cuda")[torch.from_numpy(req).cuda()]
    liked += 0.3 * torch.rand(liked.shape, generator=gen, device="cuda")
    liked.masked_fill_((torch.arange(most, device="cuda") >= blocks[:, None])[:, None], -1)
    best, at = liked.topk(min(take, most), dim=-1)
    chosen = at.masked_fill(best < 0, 1 << 30).sort(-1).values
    chosen = torch.nn.functional.pad(chosen, (0, take - chosen.shape[-1]), value=1 << 30)
    s["chosen"] = chosen.masked_fill(chosen == 1 << 30, -1).to(torch.int32).contiguous()
    s["mask"] = None
    if c["mask"] != "chain":
        nodes, words = c["nodes"], _pages(c["nodes"], 64)
        see = np.zeros((n_rows, words * 64), dtype=np.uint8)
        at = 0
        for n in rows:
            for i in range(n):
                if c["mask"] == "full":
                    see[at + i, :n] = 1
                else:  # a tree in the order its nodes were drafted: a node sees itself and its ancestors
                    see[at + i] = see[at + rnd.randint(max(0, i - 12), i)] if i else 0
                    see[at + i, i] = 1
            at += n
        s["mask"] = torch.from_numpy(np.packbits(see, axis=-1, bitorder="little").view(np.int64)).cuda()
    return s


# --- the framework's calls ---


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s)
    return {"fork": _fork_life, "resize": _churn, "compact": _pack, "bounds": _bounds, "select": _select, "sparse": _sparse}[op](s, PLAIN)


def _run_own(s):
    import block_draft_proposal_amd as D

    c = s["case"]
    if "own" not in s:  # the handles and the workspaces that a server keeps
        s["own"] = True
        if "refs" in s:
            s["pool"] = D.KVPool(s["refs"], c["page"])
            s["workspace"] = torch.empty(D.kv_pages_workspace_size(s["pool"], n_req=s["table"].shape[0], table_width=s["table"].shape[1]), dtype=torch.uint8, device="cuda")
            s["caches"] = [D.KVCache(x["k"], x["v"], x["k_scale"], x["v_scale"]) for x in s.get("layers", [])]
        if "low_high" in s:
            s["bounds"] = D.KVBounds(s["low_high"], s["unit"], page_size=c["page"])
        if c["op"] in ("bounds", "sparse"):
            s["cache"] = D.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if c["op"] == "select":
            size = D.kv_select_workspace_size(s["bounds"], n_rows=s["n_rows"], table_width=s["table"].shape[1])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        if c["op"] == "sparse":
            size = D.sparse_attention_workspace_size(s["cache"], n_rows=s["n_rows"], n_take=c["take"], max_nodes=c["nodes"], n_q_heads=c["hq"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if c["op"] == "bounds":
        D.dflash_kv_bounds(s["cache"], s["bounds"], page_table=s["table"], start=s["start"], end=s["end"])
        return s["low_high"], s["unit"]
    if c["op"] in ("select", "sparse"):
        batch = dict(page_table=s["table"], start=s["start"], offsets=s["offsets"], workspace=s["workspace"])
        if c["op"] == "select":
            return D.dflash_kv_select(s["q"], s["bounds"], max_nodes=c["nodes"], out=s["chosen"], **batch)
        return D.dflash_sparse_attention(s["q"], s["cache"], s["chosen"], max_nodes=c["nodes"], mask=s["mask"], scale=s["scale"], out=s["out"], **batch)
    rows = dict(page_table=s["table"], lens=s["lens"], workspace=s["workspace"])
    calls = dict(
        resize=lambda want: D.dflash_kv_resize(s["pool"], want=want, copies=s["copies"], counts=s["counts"], **rows),
        fork=lambda: D.dflash_kv_fork(s["pool"], parents=s["parents"], **rows),
        compact=lambda: D.dflash_kv_compact(s["pool"], copies=s["copies"], counts=s["counts"], page_map=s["map"], **rows),
        copy=lambda: [D.dflash_kv_copy_pages(cache, s["copies"], s["counts"]) for cache in s["caches"]],
    )
    return {"fork": _fork_life, "resize": _churn, "compact": _pack}[c["op"]](s, calls)


def _books_of(s):
    return {name: s[name] for name in ("refs", "table", "lens", "copies", "counts", "map") if name in s}


def _contents(s):
    return [{name: x[name] for name in ("k", "v", "k_scale", "v_scale") if x[name] is not None} for x in s["layers"]]


def _fork_life(s, calls):
    """Beams are reordered and grow; samples are let go, forked anew and grow. What has to be copied is."""
    calls = calls(s) if callable(calls) else calls
    if s["case"]["life"] == "samples":
        calls["resize"](s["wants"][0])
    calls["fork"]()
    calls["resize"](s["wants"][s["turn"] % 8 if s["case"]["life"] == "beams" else 1])
    calls["copy"]()
    s["turn"] += 1
    return _books_of(s), _contents(s)


def _churn(s, calls):
    """One half of the requests ends and the other begins."""
    calls = calls(s) if callable(calls) else calls
    calls["resize"](s["wants"][s["turn"] % 2])
    s["turn"] += 1
    return _books_of(s)


def _pack(s, calls):
    """One half of the requests ends, the pool is packed, and the half begins anew."""
    calls = calls(s) if callable(calls) else calls
    calls["resize"](s["wants"][s["turn"] % 2])
    calls["compact"]()
    calls["copy"]()
    packed = s["counts"].clone()
    calls["resize"](s["wants"][2])
    s["turn"] += 1
    return _books_of(s), _contents(s), packed


# --- the plain forms ---


def PLAIN(s):
    return dict(resize=lambda want: _resize(s, want), fork=lambda: _fork(s), compact=lambda: _compact(s), copy=lambda: _copy(s))


def _hold(refs, pages, by):
    refs.index_add_(0, pages.long().flatten(), torch.full((pages.numel(),), by, dtype=refs.dtype, device=refs.device))


def _resize(s, want):
    refs, table, lens, page = s["refs"], s["table"], s["lens"], s["case"]["page"]
    n, width = table.shape
    row, col = torch.arange(n, device="cuda"), torch.arange(width, device="cuda")
    has, needs = (_pages(x.long(), page) for x in (lens, want))
    gone = (col < has[:, None]) & (col >= needs[:, None])
    _hold(refs, table[gone], -1)
    table[gone] = -1
    lens.copy_(torch.minimum(lens, want))
    grows = want > lens
    # copies: the last page is partly filled, and others hold it who do not all grow
    last = table.gather(1, (has - 1).clamp(min=0)[:, None])[:, 0].long().clamp(min=0)
    part = grows & (lens % page != 0)
    growing = torch.zeros_like(refs).index_add_(0, last[part], torch.ones_like(refs[last[part]]))
    first = torch.full((refs.numel(),), n, device="cuda").scatter_reduce_(0, last[part], row[part], "amin")
    copy = part & (refs[last] > 1) & ~((growing[last] == refs[last]) & (first[last] == row))
    more = torch.where(grows, needs - has, 0) + copy
    begin = more.cumsum(0) - more
    free = (refs == 0).nonzero()[:, 0]
    short = int(more.sum()) - free.numel()
    if short > 0:
        s["counts"].copy_(torch.tensor([0, short]))
        return
    new = free[begin[copy]]
    pairs = torch.stack([last[copy], new], dim=1).int()
    s["copies"][: pairs.shape[0]] = pairs
    _hold(refs, pairs[:, 0], -1)
    table[row[copy], has[copy] - 1] = pairs[:, 1]
    fresh = (col >= has[:, None]) & (col < needs[:, None]) & grows[:, None]
    table[fresh] = free[(begin[:, None] + copy[:, None] + col - has[:, None])[fresh]].int()
    refs[free[: int(more.sum())]] = 1
    lens.copy_(want)
    s["counts"].copy_(torch.stack([copy.sum(), torch.zeros_like(copy.sum())]))


def _fork(s):
    refs, table, lens, page, parents = s["refs"], s["table"], s["lens"], s["case"]["page"], s["parents"].long()
    col = torch.arange(table.shape[1], device="cuda")
    others = parents != torch.arange(table.shape[0], device="cuda")
    before = col < _pages(lens.long(), page)[:, None]
    _hold(refs, table[before & others[:, None]], -1)
    table.copy_(torch.where(before, table, -1)[parents])
    lens.copy_(lens[parents])
    after = col < _pages(lens.long(), page)[:, None]
    _hold(refs, table[after & others[:, None]], 1)


def _compact(s):
    refs, table, page = s["refs"], s["table"], s["case"]["page"]
    n = refs.numel()
    used, free = (refs > 0).nonzero()[:, 0].flip(0), (refs == 0).nonzero()[:, 0]
    m = min(used.numel(), free.numel(), s["copies"].shape[0])
    src, dst = used[:m], free[:m]
    src, dst = src[src > dst], dst[src > dst]
    page_map = torch.where(refs != 0, torch.arange(n, device="cuda"), -1)
    page_map[src] = dst
    s["copies"][: src.numel()] = torch.stack([src, dst], dim=1).int()
    s["counts"].copy_(torch.tensor([src.numel(), used.numel()]))
    refs[dst] = refs[src]
    refs[src] = 0
    s["map"].copy_(page_map)
    held = torch.arange(table.shape[1], device="cuda") < _pages(s["lens"].long(), page)[:, None]
    table[held] = page_map[table[held].long()].int()


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t  # indexing has no form for 8-bit floats


def _copy(s):
    live = torch.arange(s["copies"].shape[0], device="cuda") < s["counts"][0]
    src, dst = s["copies"][live].long().unbind(1)
    for layer in _contents(s):
        for t in layer.values():
            _bytes(t)[dst] = _bytes(t)[src]


def _values(codes, scale, kind):
    x = codes.view(TYPES[kind]).float()
    return x if kind == "bf16" else torch.ldexp(x, scale.int()[..., None] - 127)


def _bounds(s, _):
    page, start, end = s["case"]["page"], s["start"].long(), s["end"].long()
    col = torch.arange(s["table"].shape[1], device="cuda")
    full = (col >= start[:, None] // page) & (col < end[:, None] // page)
    at = s["table"][full].long()
    k = _values(_bytes(s["k"])[at], None if s["k_scale"] is None else s["k_scale"][at], s["case"]["type"])
    low, high = k.amin(2), k.amax(2)
    top = torch.maximum(low.abs(), high.abs()).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - 7 + (m > 127 / 128), -100).clamp(min=-100)
    both = torch.stack([torch.ldexp(low, -e[..., None]).floor(), torch.ldexp(high, -e[..., None]).ceil()], dim=2)
    s["low_high"][at] = both.to(torch.int8)
    s["unit"][at] = (e + 127).to(torch.uint8)
    return s["low_high"], s["unit"]


def _rows_of(s):
    """(row, request, node) of every row of the ragged batch, the padding left out."""
    offsets = s["offsets"].long()
    row = torch.arange(s["n_rows"], device="cuda")
    req = torch.searchsorted(offsets[1:], row, right=True)
    live = req < len(offsets) - 1
    row, req = row[live], req[live]
    return row, req, row - offsets[req]


def _select(s, _):
    c = s["case"]
    n, nodes, hkv, dim, take, page = c["n_req"], c["nodes"], c["hkv"], c["dim"], c["take"], c["page"]
    row, req, node = _rows_of(s)
    blocks = s["start"].long() // page
    most = max(1, int(c["prefix"]) // page)
    at = s["table"][:, :most].long().clamp(min=0)
    # queries to 8 bits, one power of two for a row's heads of one kv head; the negative part goes with the least keys
    q = torch.zeros((n, nodes, c["hq"], dim), device="cuda")
    q[req, node] = s["q"][row].float()
    q = q.view(n, nodes, hkv, -1, dim)
    top = q.abs().amax((-1, -2))
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - 7 + (m > 127 / 128), -100).clamp(min=-100)
    q = torch.ldexp(q, -e[..., None, None]).round()
    q = torch.cat([q.clamp(max=0), q.clamp(min=0)], dim=-1).transpose(1, 2).reshape(n * hkv, -1, 2 * dim)
    edges = s["low_high"][at].permute(0, 2, 3, 4, 1).reshape(n * hkv, 2 * dim, most).float()
    score = (q @ edges).view(n, hkv, nodes, -1, most).amax(3)  # whole numbers below 2^24: exact
    score = torch.ldexp(score, s["unit"][at].int().permute(0, 2, 1)[:, :, None] - 147)
    col = torch.arange(most, device="cuda")
    count = blocks[:, None, None, None]
    score = torch.where((col < 1) | (col >= count - 1), math.inf, score).masked_fill(col >= count, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :take]
    order = order.masked_fill(order >= count, 1 << 30).sort(-1).values
    order = order.masked_fill(order == 1 << 30, -1).transpose(1, 2)
    s["chosen"][row, :, : order.shape[-1]] = order[req, node].int()
    return s["chosen"]


def _sparse(s, _):
    c = s["case"]
    hkv, page, group, kind = c["hkv"], c["page"], c["hq"] // c["hkv"], c["type"]
    row, req, node = _rows_of(s)
    start, table = s["start"].long()[req], s["table"][req]
    count = (s["offsets"][1:] - s["offsets"][:-1]).long()[req]
    # positions [row, kv head, key]: the chosen pages', then those behind the last full page
    chosen = s["chosen"][row].long()
    near = (chosen[..., None] * page + torch.arange(page, device="cuda")).flatten(2)
    rest = (start // page * page)[:, None] + torch.arange(page + c["nodes"], device="cuda")
    j = rest - start[:, None]
    if s["mask"] is None:
        see = j <= node[:, None]
    else:
        at = j.clamp(0, c["nodes"] - 1)
        see = (j < 0) | ((s["mask"][row].gather(1, at // 64) >> (at % 64)) & 1).bool()
    see = see & (j < count[:, None])
    pos = torch.cat([near, rest[:, None].expand(-1, hkv, -1)], dim=-1)
    see = torch.cat([near >= 0, see[:, None].expand(-1, hkv, -1)], dim=-1)
    pos = pos.masked_fill(~see, 0)
    pg = table[:, None].expand(-1, hkv, -1).gather(2, pos // page).long().clamp(min=0)
    head, slot = torch.arange(hkv, device="cuda")[:, None], pos % page

    def rows(name):  # [row, kv head, key, dim] in fp32
        scale = None if s[name + "_scale"] is None else s[name + "_scale"][pg, head, slot]
        return _values(_bytes(s[name])[pg, head, slot], scale, kind)

    q = s["q"][row].float().view(len(row), hkv, group, -1)
    score = (q @ rows("k").transpose(2, 3)).mul_(s["scale"]).masked_fill_(~see[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == -math.inf, 0)).exp_()
    out = (p @ rows("v")) / p.sum(-1, keepdim=True)
    s["out"][row] = out.masked_fill(top == -math.inf, 0).flatten(1, 2).view(len(row), c["hq"], -1).to(torch.bfloat16)
    return s["out"]


# --- attention from its definition, one row after the other, in 64 bits; the other operators' outputs are whole numbers ---


def exact(case, seed):
    if case["op"] != "sparse":
        return None
    s = prepare(case, seed)
    start, rows = _batch(case)
    if int(rows.sum()) * case["hkv"] > 8192:
        return None
    page, group = case["page"], case["hq"] // case["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    chosen = s["chosen"].cpu().numpy()
    bits = None if s["mask"] is None else np.unpackbits(s["mask"].cpu().numpy().view(np.uint8), axis=-1, bitorder="little")

    def context(name, r, head, pos):
        pg = s["table"][r].long()[pos // page]
        codes = _bytes(s[name])[pg, head, pos % page].view(TYPES[case["type"]]).float().double()
        if s[name + "_scale"] is None:
            return codes
        return codes * torch.exp2(s[name + "_scale"][pg, head, pos % page].double() - 127)[:, None]

    i = 0
    for r in range(case["n_req"]):
        a, n = int(start[r]), int(rows[r])
        for node in range(n):
            nodes = np.arange(n)[: node + 1] if bits is None else np.nonzero(bits[i, :n])[0]
            for head in range(case["hkv"]):
                ids = chosen[i, head]
                pos = [np.arange(x * page, x * page + page) for x in ids[ids >= 0].tolist()]
                pos = torch.from_numpy(np.concatenate(pos + [np.arange(a // page * page, a), a + nodes]).astype(np.int64)).cuda()
                if not len(pos):
                    continue
                at = slice(head * group, (head + 1) * group)
                w = torch.softmax(s["q"][i, at].double() @ context("k", r, head, pos).T.contiguous() * s["scale"], dim=-1)
                out[i, at] = w @ context("v", r, head, pos)
            i += 1
    return out
