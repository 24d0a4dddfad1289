"""Cases and plain forms of the operators on pages that sequences share.

The cache is that of operators.py: K and V pools of pages, a table of page
numbers per sequence, the sequences' lengths.  Here several sequences may name
the same page, and a page's count says how many table entries do.

  shared   one new token of every sequence attends over its cached tokens, where
           the sequences of a group have their first tokens in common
  fork     every sequence becomes a copy of another (its pages named once more), or is freed;
           where all are samples of one prompt, those of the prompt before end first
  resize   drafts are given back and room for the next ones is made: pages freed, pages taken
  beams    a beam search's step: fork, then room for a token each, for which a
           page that several name is copied in all layers
  compact  the table is put back as it was, its pages are counted and the pages in use moved
           to the front of the pools of all layers
  copy     pages go to other pages of another cache, all layers

``run`` computes them with elementary torch operations, or, where ``own`` is
true, by the framework's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # four beams of a short prompt: nothing but latency
        dict(name="shared_beams_4x509", op="shared", batch=4, groups=1, prefix=509, prefixes="same", rest=37,
             heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", layout="nhd", short=False),
        # a batch behind one long system prompt: 512 query rows a KV head, the largest product
        dict(name="shared_system_64x32768", op="shared", batch=64, groups=1, prefix=32768, prefixes="same", rest=2048,
             heads=64, kv_heads=8, dim=128, page=64, dtype="bf16", layout="hnd", short=False),
        # many prompts, each sampled up to eight times; some sequences ended, some prompts short
        dict(name="shared_ragged_24_groups", op="shared", batch=96, groups=24, prefix=8192, prefixes="ragged", rest=700,
             heads=32, kv_heads=8, dim=64, page=16, dtype="fp16", layout="nhd", short=True),
        # one KV head for all query heads, wide heads, a page size that no tile divides
        dict(name="shared_one_head", op="shared", batch=12, groups=2, prefix=5001, prefixes="ragged", rest=300,
             heads=24, kv_heads=1, dim=256, page=24, dtype="fp16", layout="nhd", short=False),
        # a beam search's choice: 16 requests of 4 beams, one of them over
        dict(name="fork_beams_16x4", op="fork", batch=64, longest=2048, beams=4, page=16),
        # one prompt of 32768 tokens sampled 64 times
        dict(name="fork_prompt_64", op="fork", batch=64, longest=32768, beams=64, page=16),
        # speculative decoding: 64 sequences give back their drafts and take room for 8 new ones
        dict(name="resize_drafts_64", op="resize", batch=64, longest=8192, more=8, page=16),
        # a beam search's step with the copies of the beams' last pages in 16 layers
        dict(name="beams_16x4", op="beams", batch=64, longest=1024, beams=4, page=16, layers=16, kv_heads=8, dim=128,
             dtype="bf16", layout="nhd"),
        # a small pool after some sequences have left it
        dict(name="compact_small", op="compact", batch=4, longest=200, page=16, fill=0.6, layers=1, kv_heads=2, dim=64,
             dtype="fp16", layout="nhd"),
        # 2 GiB in four layers, half of the pages in use
        dict(name="compact_2gib", op="compact", batch=40, longest=3328, page=16, fill=0.5, layers=4, kv_heads=8, dim=128,
             dtype="bf16", layout="hnd"),
        # a short sequence's pages go to another cache, 32 layers
        dict(name="copy_few", op="copy", pages=19, page=16, layers=32, kv_heads=8, dim=128, dtype="bf16", layout="nhd",
             to_layout="nhd"),
        # 32768 tokens of four layers to a cache that is stored the other way
        dict(name="copy_32768", op="copy", pages=512, page=64, layers=4, kv_heads=8, dim=128, dtype="bf16", layout="nhd",
             to_layout="hnd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "shared", "fork", "resize", "beams", "compact", "copy"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 7])
    c = dict(op=op, page=page)
    if op not in ("fork", "resize"):
        c.update(kv_heads=rng.choice([1, 2, 4, 8, 8, 16]), dim=rng.choice([64, 128, 128, 256, 80, 96, 192]),
                 dtype=rng.choice(["bf16", "bf16", "fp16"]), layout=rng.choice(["nhd", "hnd"]))
    if op == "shared":
        kvh, dim = c["kv_heads"], c["dim"]
        group = rng.choice([1, 2, 3, 4, 4, 7, 8, 12, 16, 32] if kvh < 16 else [1, 2, 4, 5])
        batch, prefix, rest = _log(rng, 1, 128), _log(rng, 1, 32768), _log(rng, 1, 4096)
        groups = min(batch, _log(rng, 1, 32))
        # no more products than the largest listed case, half of its K and V at most
        while (batch * group * kvh * dim * (prefix + rest) > 1 << 33 or (batch * rest + groups * prefix) * kvh * dim > 1 << 27
               or batch * group * kvh * prefix > 1 << 28):
            batch, prefix, rest = max(1, batch * 3 // 4), max(1, prefix * 3 // 4), max(1, rest * 3 // 4)
            groups = min(groups, batch)
        c.update(batch=batch, groups=groups, prefix=prefix, rest=rest, heads=kvh * group, short=rng.random() < 0.3,
                 prefixes=rng.choice(["same", "ragged"]))
    elif op in ("fork", "resize"):
        c.update(batch=_log(rng, 1, 256), longest=_log(rng, 1, 16384))
        if op == "fork":
            c["beams"] = rng.choice([1, 2, 4, 5, 8, c["batch"]])
        else:
            c["more"] = _log(rng, 1, 256)
    elif op == "beams":
        c.update(batch=_log(rng, 1, 64), longest=_log(rng, 1, 1024), beams=rng.choice([2, 4, 5, 8]), layers=rng.choice([1, 2, 5, 16]))
        while c["batch"] * (c["longest"] + page) * c["layers"] * c["kv_heads"] * c["dim"] > 1 << 29:
            c["longest"] = max(1, c["longest"] // 2)
            c["layers"] = max(1, c["layers"] - 1)
    elif op == "compact":
        c.update(batch=_log(rng, 1, 64), longest=_log(rng, 1, 4096), fill=rng.choice([0.2, 0.5, 0.8, 0.95, 1.0]),
                 layers=rng.choice([1, 2, 4]))
        while c["batch"] * (c["longest"] / c["fill"] + page) * c["layers"] * c["kv_heads"] * c["dim"] > 1 << 29:
            c["longest"] = max(1, c["longest"] // 2)
            c["batch"] = max(1, c["batch"] * 3 // 4)
    else:
        c.update(pages=_log(rng, 1, 2048), layers=rng.choice([1, 2, 7, 32]), to_layout=rng.choice(["nhd", "hnd"]))
        while c["pages"] * page * c["layers"] * c["kv_heads"] * c["dim"] > 1 << 27:
            c["pages"] = max(1, c["pages"] // 2)
            c["layers"] = max(1, c["layers"] * 3 // 4)
    return c


# --- what a case is, without its data: fixed lists, so that its work is known ----------------------------------------


def _groups(case):
    """Sizes of the groups, tokens that each has in common, and the sequences' lengths."""
    batch, groups = case["batch"], case["groups"]
    rng = random.Random(batch * 1000003 + groups * 101 + case["prefix"])
    sizes = [batch // groups + (g < batch % groups) for g in range(groups)]
    if case["prefixes"] == "ragged":
        for _ in range(groups):         # some groups are larger than others
            a, b = rng.randrange(groups), rng.randrange(groups)
            if sizes[a] > 1:
                sizes[a] -= 1
                sizes[b] += 1
        shared = [min(case["prefix"], _log(rng, 1, case["prefix"] + 1)) for _ in sizes]
        shared[0] = case["prefix"]
        if groups > 4:
            shared[3] = 0
    else:
        shared = [case["prefix"]] * groups
    lens = []
    for size, common in zip(sizes, shared):
        for i in range(size):
            n = common + _log(rng, 1, case["rest"] + 1) - 1
            if case["short"] and i and rng.random() < 0.2:
                n = rng.choice([0, min(common // 2, case["rest"])])      # ended, or begun again elsewhere
            lens.append(n)
    return sizes, shared, lens


def _lens(case):
    rng = random.Random(case["batch"] * 1000003 + case["longest"])
    beams = case.get("beams", 1)
    lens = []
    while len(lens) < case["batch"]:
        lens += [min(case["longest"], _log(rng, max(1, case["longest"] // 8), case["longest"] + 1))] * beams
    lens = lens[:case["batch"]]
    if beams == 1 and case["batch"] > 3:
        lens[2], lens[3] = 0, 1
    if beams >= case["batch"]:
        lens = [case["longest"]] * case["batch"]
    return lens


def _parents(case):
    """Every sequence's parent: one of its request (in a fork alone, in half of the requests, each of another); all of
    one prompt; -1 where a request is over."""
    batch, beams = case["batch"], case["beams"]
    if beams >= batch:
        return [0] * batch
    rng = random.Random(batch * 77 + beams)
    parents = []
    for first in range(0, batch, beams):
        size = min(beams, batch - first)
        turn = rng.randrange(size)
        for i in range(size):
            other = (i + turn) % size if case["op"] == "fork" and first // beams % 2 else rng.randrange(size)
            parents.append(first + other)
    if case["op"] == "fork" and batch >= 4 * beams:
        parents[2 * beams:3 * beams] = [-1] * beams
    return parents


def _held(case, lens):
    return [-(-n // case["page"]) for n in lens]


def _width(case):
    most = max(_lens(case)) + case.get("more", 1)
    return -(-most // case["page"])


def _spare(case, lens):
    """Pages that no sequence has at the start."""
    if case["op"] == "compact":
        used = sum(_held(case, lens))
        return int(used / case["fill"]) - used
    return case["batch"] * (case.get("more", 1) // case["page"] + 2) + 5


def _token_bytes(case):
    return 2 * 2 * case["kv_heads"] * case["dim"]


def work(case):
    op, page = case["op"], case["page"]
    if op == "shared":
        sizes, shared, lens = _groups(case)
        tokens, rows, pages, b = 0, 0, 0, 0
        for size, common in zip(sizes, shared):
            tokens += common
            pages += -(-common // page)
            for n in lens[b:b + size]:
                apart = n - common if n >= common else n
                tokens += apart
                pages += -(-apart // page)
                rows += n
            b += size
        per = case["batch"] * case["heads"]
        bytes_ = tokens * _token_bytes(case) + 2 * per * case["dim"] * 2 + 4 * per + 4 * pages
        return {"bytes": bytes_ + 8 * case["batch"], "flops": 4 * rows * case["heads"] * case["dim"]}
    if op == "copy":
        return {"bytes": 2 * case["pages"] * page * case["layers"] * _token_bytes(case) + 8 * case["pages"], "flops": 0}
    lens = _lens(case)
    held = _held(case, lens)
    if op == "compact":
        used = sum(held)
        pages = used + _spare(case, lens)
        moved = used * (pages - used) // pages           # what a random order leaves behind the front
        bytes_ = 4 * 3 * sum(held) + 4 * 2 * pages       # the table put back, counted and renamed; the counts
        return {"bytes": bytes_ + 2 * moved * page * case["layers"] * _token_bytes(case), "flops": 0}
    if op == "resize":
        fresh = sum(-(-(n + case["more"]) // page) - h for n, h in zip(lens, held))
        return {"bytes": 2 * fresh * (4 + 8) + 16 * case["batch"], "flops": 0}
    parents = _parents(case)
    names = sum(held[p] if p >= 0 else 0 for b, p in enumerate(parents) if p != b)
    old = sum(held[b] for b, p in enumerate(parents) if p != b)
    if op == "fork" and case["beams"] >= case["batch"]:
        names += old                                     # freed, and named again
    bytes_ = 4 * 2 * names + 8 * (names + old) + 12 * case["batch"]
    if op == "beams":
        for first in set(parents):
            several = parents.count(first)               # all but one of them take a copy of the slots in use
            if several > 1:
                bytes_ += (several - 1) * 2 * (lens[first] % page) * case["layers"] * _token_bytes(case)
    return {"bytes": bytes_, "flops": 0}


# --- inputs ---------------------------------------------------------------------------------------------------------


class _State:
    pass


def _pools(case, pages, gen, dev, layout=None, fill=True):
    """[layers, K and V, pages, kv_heads, page, dim]: N(0, 1) with 4 outlier channels a KV head in K, as a cache has them."""
    kvh, dim, page, dt = case["kv_heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    layers = case.get("layers", 1)
    if (layout or case["layout"]) == "hnd":
        kv = torch.zeros(layers, 2, pages, kvh, page, dim, dtype=dt, device=dev)
    else:
        kv = torch.zeros(layers, 2, pages, page, kvh, dim, dtype=dt, device=dev).transpose(3, 4)
    if fill:
        loud = torch.ones(2, 1, kvh, 1, dim, dtype=torch.float32, device=dev)
        for h in range(kvh):
            loud[0, 0, h, 0, torch.randperm(dim, generator=gen, device=dev)[:4]] = 8.0
        step = max(1, (1 << 27) // (2 * kvh * page * dim))
        for i in range(layers):
            for p in range(0, pages, step):
                shape = kv[i, :, p:p + step].shape
                kv[i, :, p:p + step] = torch.randn(shape, generator=gen, device=dev) * loud
    return kv


def _table(held, width, spare, gen, dev):
    """Pages of every sequence in a random order of the pool, -1 behind them, and the pool's size."""
    total = sum(held) + spare
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(held), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 13)
    st = _State()
    st.case, st.page = case, case["page"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if case["op"] == "copy":
        n = case["pages"]
        st.kv = _pools(case, n + 5, gen, dev)
        st.to = _pools(case, n + 9, gen, dev, case["to_layout"], fill=False)
        st.src = torch.randperm(n + 5, generator=gen, device=dev)[:n].to(torch.int32)
        st.dst = torch.randperm(n + 9, generator=gen, device=dev)[:n].to(torch.int32)
        return st
    if case["op"] == "shared":
        st.sizes, st.host_shared, st.host_lens = sizes, shared, lens = _groups(case)
        firsts = [sum(sizes[:g]) for g in range(len(sizes) + 1)]
        st.cu, st.shared, st.lens = ints(firsts), ints(shared), ints(lens)
        # the pages of a group's first sequence stand in the tables of its others as far as they are full
        held = _held(case, lens)
        full = [0] * len(lens)
        for first, size, common in zip(firsts, sizes, shared):
            for b in range(first + 1, first + size):
                full[b] = min(common, lens[b]) // st.page
        part, pages = _table([h - f for h, f in zip(held, full)], max(held + [1]), 3, gen, dev)
        st.table = torch.full_like(part, -1)
        edges = []
        for first, size, common in zip(firsts, sizes, shared):
            for b in range(first, first + size):
                f = full[b]
                st.table[b, f:held[b]] = part[b, :held[b] - f]
                st.table[b, :f] = st.table[first, :f]
                if b > first and min(common, lens[b]) % st.page:
                    edges.append((first, b, f))
        st.kv = _pools(case, pages, gen, dev)
        if edges:           # the tokens in common of a page that is not full of them: each its own copy
            a, b, i = (torch.tensor(e, device=dev) for e in zip(*edges))
            st.kv[:, :, st.table[b, i].long()] = st.kv[:, :, st.table[a, i].long()]
        st.q = torch.randn(case["batch"], case["heads"], case["dim"], generator=gen, device=dev).to(DTYPES[case["dtype"]])
        st.scale = 1.0 / math.sqrt(case["dim"])
        return st
    lens = _lens(case)
    held = _held(case, lens)
    st.table, pages = _table(held, _width(case), _spare(case, lens), gen, dev)
    st.lens = ints(lens)
    st.base, st.longer = ints(lens), ints([n + case.get("more", 1) for n in lens])
    st.width, st.refs = _width(case), None
    if "beams" in case:
        st.parents = ints(_parents(case))
        st.over = ints([b if case["beams"] < case["batch"] or b == 0 else -1 for b in range(case["batch"])])
    if "dim" in case:
        st.kv = _pools(case, pages, gen, dev)
    else:           # pages that nothing reads: the smallest there are
        st.kv = torch.zeros(1, 2, pages, 1, st.page, 8, dtype=torch.bfloat16, device=dev)
    st.scattered = st.table.clone()
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import lossless_bf16_tensor_splitzip_amd as S

        if case["op"] == "copy":
            none = torch.zeros(0, 0, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
            st.pages, st.to_pages = (S.KVPages([S.KVCache(k, v, *none) for k, v in kv]) for kv in (st.kv, st.to))
        elif case["op"] == "shared":
            st.cache = S.KVCache(st.kv[0, 0], st.kv[0, 1], st.table, st.lens)
            st.ws = S.KVSharedWorkspace(st.cache, case["heads"], case["groups"])
            st.out = torch.empty_like(st.q)
            st.lse = torch.empty(case["batch"], case["heads"], device="cuda")
        else:
            st.pages = S.KVPages([S.KVCache(k, v, st.table, st.lens) for k, v in st.kv])
            st.pages.count()
            st.refs = st.pages.refs
            st.moved = torch.empty(st.kv.shape[2], dtype=torch.int32, device="cuda")
            st.used = torch.empty(1, dtype=torch.int32, device="cuda")
    elif case["op"] not in ("copy", "shared"):
        st.refs = _count(st.table, st.kv.shape[2])
    return st


# --- the framework's calls ------------------------------------------------------------------------------------------


def _run_own(st):
    op = st.case["op"]
    if op == "shared":
        st.cache.attend_shared(st.q, st.cu, st.shared, st.ws, out=st.out, scale=st.scale, lse=st.lse)
        return st.out, st.lse
    if op == "copy":
        st.pages.copy(st.src, st.dst, to=st.to_pages)
        return st.to
    if op == "fork":
        if st.case["beams"] >= st.case["batch"]:
            st.pages.fork(st.over)
        st.pages.fork(st.parents)
        return st.table, st.lens, st.refs
    if op == "resize":
        st.pages.resize(st.base)
        st.pages.resize(st.longer)
        return st.table, st.lens, st.refs
    if op == "beams":
        st.pages.resize(st.base)
        st.pages.fork(st.parents)
        st.pages.resize(st.longer)
        return st.table, st.lens, st.refs, st.kv
    st.table.copy_(st.scattered)
    st.pages.count()
    st.pages.compact(moved=st.moved, used=st.used)
    return st.table, st.refs, st.kv, st.moved, st.used


# --- the plain forms ------------------------------------------------------------------------------------------------


def _count(table, pages):
    """How many entries name each page."""
    refs = torch.zeros(pages + 1, dtype=torch.int32, device=table.device)
    at = torch.where(table >= 0, table, pages).long().reshape(-1)
    return refs.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:pages].contiguous()


def _fork(st, parents):
    take = parents.clamp(min=0).long()
    over = parents < 0
    st.table.copy_(torch.where(over[:, None], -1, st.table[take]))
    st.lens.copy_(torch.where(over, 0, st.lens[take]))
    st.refs.copy_(_count(st.table, st.refs.numel()))


def _resize(st, lens):
    page, pages, dev = st.page, st.refs.numel(), st.table.device
    batch, width = st.table.shape
    need = (lens + page - 1) // page
    column = torch.arange(width, device=dev)
    st.table.masked_fill_(column >= need[:, None], -1)
    refs = _count(st.table, pages)
    # who writes into a page that others name: the slots behind its length, in a page that is begun
    old, b = st.lens, torch.arange(batch, device=dev)
    begun = (lens > old) & (old % page != 0)
    at = (old // page).clamp(max=width - 1).long()
    x = torch.where(begun, st.table[b, at], pages).long()
    writers = torch.zeros(pages + 1, dtype=torch.int32, device=dev).index_add_(0, x, torch.ones_like(old))
    lowest = torch.full((pages + 1,), batch, device=dev).scatter_reduce_(0, x, b, "amin")
    counts = torch.cat([refs, refs.new_zeros(1)])
    copied = begun & (counts[x] > 1) & ~((writers[x] == counts[x]) & (lowest[x] == b))
    # the wanted pages in order: a sequence's copy, then its new ones
    wanted = torch.cat([copied[:, None], (column < need[:, None]) & (st.table < 0)], 1)
    rank = (torch.cumsum(wanted.reshape(-1), 0) - 1).reshape(wanted.shape)
    free = torch.nonzero(refs == 0).reshape(-1)
    given = wanted & (rank < free.numel())
    number = torch.cat([free, free.new_zeros(1)])[torch.where(given, rank, free.numel())].to(torch.int32)
    fresh = given[:, 1:]
    st.table.copy_(torch.where(fresh, number[:, 1:], st.table))
    moved = given[:, 0]
    rows = torch.nonzero(moved).reshape(-1)
    if rows.numel() and "dim" in st.case:
        source, target = x[rows], number[rows, 0].long()
        slot = torch.arange(page, device=dev) < (old[rows] % page)[:, None]
        st.kv[:, :, target] = torch.where(slot[None, None, :, None, :, None], st.kv[:, :, source], st.kv[:, :, target])
    st.table[rows, at[rows]] = number[rows, 0]
    held = need - (wanted & ~given)[:, 1:].sum(1)
    st.lens.copy_(torch.where(copied & ~moved, old, torch.minimum(lens, held * page)))
    st.refs.copy_(_count(st.table, pages))


def _compact(st):
    pages, dev = st.refs.numel(), st.table.device
    st.table.copy_(st.scattered)
    column = torch.arange(st.width, device=dev)
    st.table.masked_fill_(column >= ((st.lens + st.page - 1) // st.page)[:, None], -1)
    refs = _count(st.table, pages)
    used = (refs > 0).sum()
    p = torch.arange(pages, device=dev)
    target = torch.nonzero((refs == 0) & (p < used)).reshape(-1)
    source = torch.nonzero((refs > 0) & (p >= used)).reshape(-1).flip(0)
    moved = torch.where(refs > 0, p, -1).to(torch.int32)
    moved[source] = target.to(torch.int32)
    st.kv[:, :, target] = st.kv[:, :, source]
    st.table.copy_(torch.where(st.table >= 0, moved[st.table.clamp(min=0).long()], st.table))
    st.refs.copy_(_count(st.table, pages))
    return st.table, st.refs, st.kv, moved, used.to(torch.int32).reshape(1)


def _rows(st, table, first, most):
    """K and V in 32 bits of `most` tokens behind position first[i], for every row i of a table:
    [rows, kv_heads, most, dim] (what a row has not is some page's)."""
    t = first[:, None] + torch.arange(most, device=table.device)
    i = (t // st.page).clamp(max=table.shape[1] - 1).long()
    where, slot = torch.gather(table, 1, i).clamp(min=0).long(), t % st.page
    return [pool[where, :, slot].transpose(1, 2).float() for pool in st.kv[0]]


def _part(q, k, v, seen, scale):
    """Largest logit, sum and weighted sum of V over the tokens seen: q [n, kv_heads, rows, dim], seen [n, 1, rows, tokens]."""
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(scale).masked_fill_(~seen, -math.inf)
    top = x.max(dim=3, keepdim=True).values
    e = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    v = torch.where(seen.any(dim=2)[..., None], v, 0.0)
    return top, e.sum(dim=3, keepdim=True), torch.matmul(e, v)


def _shared(st):
    case, dev = st.case, st.q.device
    kvh, dim, batch = case["kv_heads"], case["dim"], case["batch"]
    group, largest = case["heads"] // kvh, max(st.sizes)
    g = torch.searchsorted(st.cu, torch.arange(batch, device=dev), right=True) - 1
    first = st.cu[g].long()
    common = torch.minimum(st.shared[g], st.lens[first])
    common = torch.where(st.lens >= common, common, 0)
    q = st.q.float().reshape(batch, kvh, group, dim)
    # a group's queries together over what it has in common: [groups, kv_heads, members * group, dim]
    heads = st.cu[:-1].long()
    most = max(st.host_shared + [1])
    together = torch.zeros(len(st.sizes), kvh, largest, group, dim, device=dev)
    place = torch.arange(batch, device=dev) - first
    together[g, :, place] = q
    k, v = _rows(st, st.table[heads], torch.zeros_like(heads), most)
    size = torch.minimum(st.shared, st.lens[heads])
    seen = (torch.arange(most, device=dev) < size[:, None])[:, None, None, :].expand(-1, 1, largest * group, -1)
    parts = _part(together.reshape(len(st.sizes), kvh, -1, dim), k, v, seen, st.scale)
    m0, l0, o0 = (p.reshape(len(st.sizes), kvh, largest, group, -1)[g, :, place] for p in parts)
    alone = (common == 0)[:, None, None, None]
    m0, l0, o0 = torch.where(alone, -math.inf, m0), torch.where(alone, 0.0, l0), torch.where(alone, 0.0, o0)
    # and every sequence over the rest of its own
    own_most = max([n - c if n >= c else n for n, c in zip(st.host_lens, _common(st))] + [1])
    k, v = _rows(st, st.table, common, own_most)
    seen = (torch.arange(own_most, device=dev) < (st.lens - common)[:, None])[:, None, None, :].expand(-1, 1, group, -1)
    m1, l1, o1 = _part(q, k, v, seen, st.scale)
    top = torch.maximum(m0, m1)
    at = torch.where(top == -math.inf, 0.0, top)
    w0, w1 = torch.exp(m0 - at), torch.exp(m1 - at)
    total = l0 * w0 + l1 * w1
    out = torch.where(total > 0, (o0 * w0 + o1 * w1) / total, 0.0)
    lse = at + torch.log(total)
    return out.reshape(st.q.shape).to(st.q.dtype), lse.reshape(batch, -1)


def _common(st):
    """Tokens in common, by sequence, of the lists that the program has on the host."""
    return [c for size, c in zip(st.sizes, st.host_shared) for _ in range(size)]


def run(st):
    if own:
        return _run_own(st)
    op = st.case["op"]
    if op == "shared":
        return _shared(st)
    if op == "copy":
        st.to[:, :, st.dst.long()] = st.kv[:, :, st.src.long()]
        return st.to
    if op == "compact":
        return _compact(st)
    if op in ("resize", "beams"):
        _resize(st, st.base)
    if op == "fork" and st.case["beams"] >= st.case["batch"]:
        _fork(st, st.over)
    if op in ("fork", "beams"):
        _fork(st, st.parents)
    if op in ("resize", "beams"):
        _resize(st, st.longer)
    return (st.table, st.lens, st.refs, st.kv) if op == "beams" else (st.table, st.lens, st.refs)


def exact(case, seed):
    """The attention in 64 bits, one KV head of one sequence at a time over its own table row, whoever shares it.
    The other operators' outputs are copies and whole numbers."""
    if case["op"] != "shared":
        return None
    st = _inputs(case, seed)
    kvh, group = case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.zeros(st.q.shape, dtype=torch.float64, device=st.q.device)
    lse = torch.full(st.q.shape[:2], -math.inf, dtype=torch.float64, device=st.q.device)
    for b, n in enumerate(st.host_lens):
        if n == 0:
            continue
        pos = torch.arange(n, device=st.q.device)
        where, slot = st.table[b].long()[pos // case["page"]], pos % case["page"]
        for h in range(kvh):
            rows = slice(h * group, (h + 1) * group)
            k, v = (pool[where, h, slot].double() for pool in st.kv[0])
            x = torch.mm(st.q[b, rows].double(), k.t().contiguous()) / math.sqrt(case["dim"])
            lse[b, rows] = torch.logsumexp(x, 1)
            out[b, rows] = torch.mm(torch.softmax(x, 1), v)
    return out, lse
