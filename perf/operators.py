"""Cases and plain forms of the key-value cache operators.

The operators work on a paged cache: K and V pools of pages, a table of page
numbers per sequence and the sequences' lengths.

  append  rows of new K and V go to their pages
  gather  rows of cached K and V come back as plain tensors (what the codec
          encodes when a sequence leaves the GPU)
  attend  one new token of every sequence attends over its cached tokens:
          all of them, or the last ``window`` and the first ``sinks``; on
          request the weight each token received, summed over the query heads
          of its KV head, is added to the token's mass
  evict   every KV head keeps ``budget`` tokens: the first ``sinks``, the last
          ``recent`` and those of the largest mass between them

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
        # a conversation's first tokens on one sequence: nothing but latency
        dict(name="attend_first_tokens", op="attend", batch=1, longest=37, spread="same", heads=32,
             kv_heads=8, dim=128, page=16, dtype="bf16", layout="nhd", window=0, sinks=0, mass=False),
        # one sequence as long as the streaming cache of the benchmark
        dict(name="attend_one_32768", op="attend", batch=1, longest=32768, spread="same", heads=32,
             kv_heads=8, dim=128, page=64, dtype="bf16", layout="hnd", window=0, sinks=0, mass=False),
        # an ordinary serving batch: lengths from nothing to 8192, small pages
        dict(name="attend_ragged_48", op="attend", batch=48, longest=8192, spread="ragged", heads=32,
             kv_heads=8, dim=128, page=16, dtype="bf16", layout="nhd", window=0, sinks=0, mass=False),
        # the largest: 4 GiB of K and V in one pass
        dict(name="attend_32x32768", op="attend", batch=32, longest=32768, spread="same", heads=64,
             kv_heads=8, dim=128, page=32, dtype="bf16", layout="hnd", window=0, sinks=0, mass=False),
        # streaming: a window of 1024 and 4 sinks of long sequences, one KV head per query head
        dict(name="attend_window_1024", op="attend", batch=16, longest=32768, spread="ragged", heads=16,
             kv_heads=16, dim=64, page=32, dtype="fp16", layout="nhd", window=1024, sinks=4, mass=False),
        # one KV head for all query heads, wide heads, a page size that no tile divides
        dict(name="attend_shared_head", op="attend", batch=12, longest=5001, spread="ragged", heads=24,
             kv_heads=1, dim=256, page=24, dtype="fp16", layout="nhd", window=0, sinks=0, mass=False),
        # attention that also keeps the accumulated weights an eviction needs
        dict(name="attend_mass_4096", op="attend", batch=16, longest=4096, spread="same", heads=32,
             kv_heads=8, dim=128, page=16, dtype="bf16", layout="hnd", window=0, sinks=0, mass=True),
        # the step's new tokens, one a sequence
        dict(name="append_step_64", op="append", batch=64, longest=4096, spread="ragged", new="one",
             kv_heads=8, dim=128, page=16, dtype="bf16", layout="nhd"),
        # prompts that arrive from a decode of their payload, [kv_heads, tokens, dim]
        dict(name="append_prompts", op="append", batch=6, longest=16384, spread="ragged", new="all",
             kv_heads=8, dim=128, page=16, dtype="bf16", layout="nhd"),
        # a sequence leaves the GPU: its rows in one piece for the encoder
        dict(name="gather_32768", op="gather", batch=1, longest=32768, spread="same", new="all",
             kv_heads=8, dim=128, page=64, dtype="bf16", layout="nhd"),
        # a batch at its budget: half of 4096 tokens go
        dict(name="evict_16x4096", op="evict", batch=16, longest=4096, spread="same", budget=2048, sinks=4,
             recent=512, kv_heads=8, dim=128, page=16, dtype="bf16", layout="hnd"),
        # one long sequence down to a quarter
        dict(name="evict_one_32768", op="evict", batch=1, longest=32768, spread="same", budget=8192, sinks=4,
             recent=1024, kv_heads=8, dim=128, page=64, dtype="bf16", layout="hnd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "gather", "evict"])
    dim = rng.choice([64, 128, 128, 256, 80, 96, 192])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    batch = _log(rng, 1, 64)
    longest = _log(rng, 1, 32768)
    # a drawn case holds at most a quarter of the largest listed one's tokens
    while batch * longest * kv_heads * dim > 1 << 28:
        batch, longest = max(1, batch * 2 // 3), max(1, longest * 3 // 4)
    c = dict(op=op, batch=batch, longest=longest, spread=rng.choice(["same", "ragged", "ragged"]),
             kv_heads=kv_heads, dim=dim, page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 7]),
             dtype=rng.choice(["bf16", "bf16", "fp16"]), layout=rng.choice(["nhd", "hnd"]))
    if op == "attend":
        c["heads"] = kv_heads * rng.choice([1, 2, 3, 4, 4, 7, 8, 12, 16, 32] if kv_heads < 16 else [1, 2, 4, 5])
        c["window"] = _log(rng, 1, max(longest, 2)) if rng.random() < 0.35 else 0
        c["sinks"] = rng.choice([0, 1, 4, 64]) if c["window"] else 0
        c["mass"] = rng.random() < 0.3
    elif op == "evict":
        c["budget"] = _log(rng, 1, longest)
        c["sinks"] = min(rng.choice([0, 4, 16]), c["budget"] // 3)
        c["recent"] = rng.randint(0, c["budget"] - c["sinks"])
    else:
        c["new"] = rng.choice(["one", "some", "all"])
    return c


def _lens(case):
    """The sequences' lengths: a fixed list for a case, so that its work is known without its data."""
    batch, longest = case["batch"], case["longest"]
    if case["spread"] == "same":
        return [longest] * batch
    rng = random.Random(batch * 1000003 + longest)
    lens = [min(longest, _log(rng, 1, longest + 1)) for _ in range(batch)]
    lens[0] = longest
    if batch > 3:
        lens[2], lens[3] = 0, 1
    return lens


def _new(case):
    """Rows that an append or a gather moves, per sequence."""
    lens = _lens(case)
    if case["new"] == "one":
        return [min(n, 1) for n in lens]
    if case["new"] == "some":
        return [(n * 3 + 7) // 8 for n in lens]
    return lens


def _visible(case, n):
    w, s = case["window"], case["sinks"]
    return n if w == 0 else min(n, min(w, n) + min(s, max(n - min(w, n), 0)))


def work(case):
    lens, kvh, dim, page = _lens(case), case["kv_heads"], case["dim"], case["page"]
    pages = sum(-(-n // page) for n in lens)
    if case["op"] == "attend":
        vis = sum(_visible(case, n) for n in lens)
        bytes_ = 2 * vis * kvh * dim * 2 + 2 * case["batch"] * case["heads"] * dim * 2
        bytes_ += 4 * min(pages, vis) + 4 * case["batch"]
        if case["mass"]:
            bytes_ += 2 * 4 * sum(lens) * kvh + 4 * case["batch"] * case["heads"]
        return {"bytes": bytes_, "flops": 4 * vis * case["heads"] * dim}
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        bytes_ = 4 * sum(lens) * kvh                       # the mass
        bytes_ += 2 * 4 * kept * kvh                       # kept tokens and their mass
        bytes_ += 2 * 2 * kept * kvh * dim * 2 + 4 * pages
        return {"bytes": bytes_, "flops": sum(lens) * kvh}
    rows = sum(_new(case))
    return {"bytes": 2 * 2 * rows * kvh * dim * 2 + 4 * min(pages, rows) + 8 * case["batch"], "flops": 0}


class _State:
    pass


def _pool(case, pages, dev):
    kvh, dim, page, dt = case["kv_heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    if case["layout"] == "hnd":
        return torch.zeros(pages, kvh, page, dim, dtype=dt, device=dev)
    return torch.zeros(pages, page, kvh, dim, dtype=dt, device=dev).transpose(1, 2)


def _table(lens, page, gen, dev, spare=3):
    """Pages of every sequence in a random order of the pool, and the pool's size."""
    need = [max(-(-n // page), 1) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 11)
    st = _State()
    st.case, st.host_lens = case, _lens(case)
    kvh, dim, page, dt = case["kv_heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    st.lens = torch.tensor(st.host_lens, dtype=torch.int32, device=dev)
    st.table, pages = _table(st.host_lens, page, gen, dev)
    st.k, st.v = _pool(case, pages, dev), _pool(case, pages, dev)
    if case["op"] != "append":
        # N(0, 1) with 4 outlier channels a KV head in K, as a KV cache has them
        loud = torch.ones(kvh, 1, dim, dtype=torch.float32, device=dev)
        for h in range(kvh):
            loud[h, 0, torch.randperm(dim, generator=gen, device=dev)[:4]] = 8.0
        step = max(1, (1 << 26) // (kvh * page * dim))
        for p in range(0, pages, step):
            shape = st.k[p:p + step].shape
            st.k[p:p + step] = torch.randn(shape, generator=gen, device=dev) * loud
            st.v[p:p + step] = torch.randn(shape, generator=gen, device=dev)
    width = max(st.host_lens)
    if case["op"] == "attend":
        st.q = torch.randn(case["batch"], case["heads"], dim, generator=gen, device=dev).to(dt)
        st.scale = 1.0 / math.sqrt(dim)
        if case["mass"]:
            st.mass = torch.rand(case["batch"], kvh, width, generator=gen, device=dev) ** 4
            st.mass_out = torch.zeros_like(st.mass)
    elif case["op"] == "evict":
        # heavy-tailed masses; the small ones are equal to others or zero, as far tokens' are
        m = torch.rand(case["batch"], kvh, width, generator=gen, device=dev) ** 8 * 4
        st.mass = torch.where(m < 0.01, torch.round(m * 1024) / 1024, m)
        st.mass_out = torch.zeros_like(st.mass)
        st.kept = torch.empty(case["batch"], kvh, case["budget"], dtype=torch.int32, device=dev)
        kept = [min(n, case["budget"]) for n in st.host_lens]
        st.to_table, pages = _table(kept, page, gen, dev, spare=0)
        st.to_k, st.to_v = _pool(case, pages, dev), _pool(case, pages, dev)
        st.to_lens = torch.zeros(case["batch"], dtype=torch.int32, device=dev)
    else:
        new = _new(case)
        rows = sum(new)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st.host_cu = cu
        st.cu = torch.tensor(cu, dtype=torch.int32, device=dev)
        if case["op"] == "append":
            st.new_k = torch.randn(kvh, rows, dim, generator=gen, device=dev).to(dt).transpose(0, 1)
            st.new_v = torch.randn(kvh, rows, dim, generator=gen, device=dev).to(dt).transpose(0, 1)
        else:
            st.new_k = torch.zeros(kvh, rows, dim, dtype=dt, device=dev).transpose(0, 1)
            st.new_v = torch.zeros(kvh, rows, dim, dtype=dt, device=dev).transpose(0, 1)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import lossless_bf16_tensor_splitzip_amd as S

        st.cache = S.KVCache(st.k, st.v, st.table, st.lens)
        if case["op"] == "attend":
            st.ws = S.KVWorkspace(st.cache, case["heads"], mass=case["mass"])
            st.out = torch.empty_like(st.q)
        elif case["op"] == "evict":
            st.to = S.KVCache(st.to_k, st.to_v, st.to_table, st.to_lens)
    return st


def _run_own(st):
    case = st.case
    if case["op"] == "attend":
        window, sinks = case["window"] or None, case["sinks"]
        if not case["mass"]:
            return st.cache.attend(st.q, st.ws, out=st.out, scale=st.scale, window=window, sinks=sinks)
        st.cache.attend(st.q, st.ws, out=st.out, scale=st.scale, window=window, sinks=sinks,
                        mass=st.mass, mass_out=st.mass_out)
        return st.out, st.mass_out
    if case["op"] == "evict":
        st.cache.evict(st.mass, case["budget"], sinks=case["sinks"], recent=case["recent"], to=st.to,
                       kept=st.kept, mass_out=st.mass_out)
        return st.kept, st.to_k, st.to_v, st.to_lens, st.mass_out
    if case["op"] == "append":
        st.cache.append(st.new_k, st.new_v, st.cu)
        return st.k, st.v
    st.cache.gather(st.new_k, st.new_v, st.cu)
    return st.new_k, st.new_v


def _rows(st, pool, b, n):
    """The first n cached rows of sequence b, [kv_heads, n, dim]."""
    page = st.case["page"]
    used = st.table[b, :-(-n // page)].long()
    kvh, dim = pool.shape[1], pool.shape[3]
    return pool[used].transpose(0, 1).reshape(kvh, -1, dim)[:, :n]


def _attend(st):
    case = st.case
    kvh, dim = case["kv_heads"], case["dim"]
    group = case["heads"] // kvh
    out = torch.zeros(st.q.shape, dtype=torch.float32, device=st.q.device)
    for b, n in enumerate(st.host_lens):
        mass = st.mass_out[b, :, :n] if case["mass"] else None
        if mass is not None:
            mass.copy_(st.mass[b, :, :n])
        if n == 0:
            continue
        k, v = _rows(st, st.k, b, n), _rows(st, st.v, b, n)
        if case["window"]:
            first = max(0, n - case["window"])
            s = min(case["sinks"], first)
            k, v = torch.cat([k[:, :s], k[:, first:]], 1), torch.cat([v[:, :s], v[:, first:]], 1)
        q = st.q[b].float().reshape(kvh, group, dim)
        x = torch.matmul(k.float(), q.transpose(1, 2).contiguous()) * st.scale       # [kvh, n, group]
        e = torch.exp(x - x.max(dim=1, keepdim=True).values)
        p = e / e.sum(dim=1, keepdim=True)
        out[b] = torch.matmul(p.transpose(1, 2).contiguous(), v.float()).reshape(-1, dim)
        if mass is not None:
            w = p.sum(dim=2)
            if case["window"]:
                mass[:, :s] += w[:, :s]
                mass[:, first:] += w[:, s:]
            else:
                mass += w
    out = out.to(st.q.dtype)
    return (out, st.mass_out) if case["mass"] else out


def _evict(st):
    case = st.case
    budget, sinks, recent, page = case["budget"], case["sinks"], case["recent"], case["page"]
    kvh, dim = case["kv_heads"], case["dim"]
    st.kept.fill_(-1)
    for b, n in enumerate(st.host_lens):
        m = st.mass[b, :, :n]
        st.mass_out[b, :, :n] = 0
        if n <= budget:
            idx = torch.arange(n, device=m.device).expand(kvh, n)
        else:
            take = budget - sinks - recent
            mid = torch.sort(m[:, sinks:n - recent], dim=1, descending=True, stable=True).indices[:, :take] + sinks
            keep = torch.zeros(kvh, n, dtype=torch.bool, device=m.device)
            keep[:, :sinks] = True
            keep[:, n - recent:] = True
            keep.scatter_(1, mid, True)
            idx = torch.nonzero(keep)[:, 1].reshape(kvh, budget)
        size = idx.shape[1]
        st.to_lens[b] = size
        if size == 0:
            continue
        st.kept[b, :, :size] = idx
        st.mass_out[b, :, :size] = torch.gather(m, 1, idx)
        t = torch.arange(size, device=m.device)
        to_page, to_slot = st.to_table[b].long()[t // page], t % page
        wide = idx[:, :, None].expand(kvh, size, dim)
        st.to_k[to_page, :, to_slot] = torch.gather(_rows(st, st.k, b, n), 1, wide).transpose(0, 1)
        st.to_v[to_page, :, to_slot] = torch.gather(_rows(st, st.v, b, n), 1, wide).transpose(0, 1)
    return st.kept, st.to_k, st.to_v, st.to_lens, st.mass_out


def run(st):
    if own:
        return _run_own(st)
    op = st.case["op"]
    if op == "attend":
        return _attend(st)
    if op == "evict":
        return _evict(st)
    page, rows = st.case["page"], st.host_cu[-1]
    r = torch.arange(rows, device=st.cu.device)
    b = torch.searchsorted(st.cu, r, right=True) - 1
    t = st.lens[b].long() - st.cu[b + 1] + r                  # the last new row is the last cached token
    where, slot = st.table[b, t // page].long(), t % page
    if op == "append":
        st.k[where, :, slot] = st.new_k
        st.v[where, :, slot] = st.new_v
    else:
        st.new_k.copy_(st.k[where, :, slot])
        st.new_v.copy_(st.v[where, :, slot])
    return (st.k, st.v) if op == "append" else (st.new_k, st.new_v)


def exact(case, seed):
    """The attention in 64 bits, one KV head of one sequence at a time. The other operators' outputs are
    copies and whole numbers."""
    if case["op"] != "attend":
        return None
    st = _inputs(case, seed)
    kvh, group = case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.zeros(st.q.shape, dtype=torch.float64, device=st.q.device)
    total = st.mass_out.double() if case["mass"] else None
    for b, n in enumerate(st.host_lens):
        pos = torch.arange(n, device=st.q.device)
        see = pos >= 0
        if case["window"]:
            see = (pos < case["sinks"]) | (pos > n - 1 - case["window"])
        if case["mass"]:
            total[b, :, :n] = st.mass[b, :, :n].double()
        pos = pos[see]
        if pos.numel() == 0:
            continue
        where, slot = st.table[b, (pos // case["page"])].long(), pos % case["page"]
        for h in range(kvh):
            q = st.q[b, h * group:(h + 1) * group].double()
            k, v = st.k[where, h, slot].double(), st.v[where, h, slot].double()
            logits = torch.stack([(k * row).sum(1) for row in q]) * (1.0 / math.sqrt(case["dim"]))
            w = torch.softmax(logits, 1)
            out[b, h * group:(h + 1) * group] = torch.stack([(v * row[:, None]).sum(0) for row in w])
            if case["mass"]:
                total[b, h, pos] += w.sum(0)
    return (out, total) if case["mass"] else out
