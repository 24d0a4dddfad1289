"""Plain 64-bit reference of the paged key-value cache, on the CPU, and the
caches the tests run on.  No code of the package."""
import math

import torch

# Relative rounding units: half a step of the type.
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
F32 = 2.0 ** -24
# The weights go into the product with V as a sum of two 16-bit numbers; the
# second one carries the first one's rounding error, so what is left is the
# product of the two units (fp16: no less than its subnormal step 2^-25 times
# the scale 2^-15 the largest weight is held at).
WEIGHT = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22}


class Made:
    pass


def make(lens, kv_heads, dim, page, dtype, layout="hnd", seed=0, heads=None, slack=2, fill=float("nan"),
         width=None, k_scale=1.0):
    """A cache on the CPU: pages in random order, everything that holds no
    token filled with ``fill``."""
    g = torch.Generator().manual_seed(seed)
    m = Made()
    m.lens, m.kv_heads, m.dim, m.page, m.dtype = list(lens), kv_heads, dim, page, dtype
    need = [-(-n // page) for n in lens]
    width = max(need + [1]) if width is None else width
    pages = sum(need) + slack
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    m.table = torch.full((len(lens), width), -1, dtype=torch.int32)
    shape = (pages, kv_heads, page, dim) if layout == "hnd" else (pages, page, kv_heads, dim)
    m.k, m.v = (torch.full(shape, fill, dtype=dtype) for _ in range(2))
    if layout == "nhd":
        m.k, m.v = m.k.transpose(1, 2), m.v.transpose(1, 2)
    at = 0
    for b, n in enumerate(lens):
        m.table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        t = torch.arange(n)
        where, slot = m.table[b].long()[t // page], t % page
        m.k[where, :, slot] = (torch.randn(n, kv_heads, dim, generator=g) * k_scale).to(dtype)
        m.v[where, :, slot] = torch.randn(n, kv_heads, dim, generator=g).to(dtype)
    if heads:
        m.q = torch.randn(len(lens), heads, dim, generator=g).to(dtype)
    return m


def to_gpu(m, S, dev="cuda:0"):
    """The same cache on the GPU, strides kept."""
    m.gk, m.gv = (torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=dev).copy_(t) for t in (m.k, m.v))
    m.gtable = m.table.to(dev)
    m.glens = torch.tensor(m.lens, dtype=torch.int32, device=dev)
    m.cache = S.KVCache(m.gk, m.gv, m.gtable, m.glens)
    if hasattr(m, "q"):
        m.gq = m.q.to(dev)
    return m


def rows(m, b, pos, pool):
    pos = torch.as_tensor(pos, dtype=torch.long)
    return pool[m.table[b].long()[pos // m.page], :, pos % m.page]      # [n, kv_heads, dim]


def visible(n, window, sinks):
    return [t for t in range(n) if window is None or t >= n - window or t < sinks]


def attend(m, scale=None, window=None, sinks=0, hidden=()):
    """Per sequence: out [heads, dim], lse [heads], weight [kv_heads, len] and
    error bounds of the three.  ``hidden``: (sequence, position) left out."""
    scale = m.dim ** -0.5 if scale is None else scale
    heads = m.q.shape[1]
    group = heads // m.kv_heads
    res = []
    for b, n in enumerate(m.lens):
        out, out_tol = torch.zeros(heads, m.dim, dtype=torch.float64), torch.zeros(heads, m.dim, dtype=torch.float64)
        lse, lse_tol = torch.full((heads,), -math.inf, dtype=torch.float64), torch.zeros(heads, dtype=torch.float64)
        w, w_tol = torch.zeros(m.kv_heads, n, dtype=torch.float64), torch.zeros(m.kv_heads, n, dtype=torch.float64)
        pos = [t for t in visible(n, window, sinks) if (b, t) not in hidden]
        if pos:
            k, v = rows(m, b, pos, m.k).double(), rows(m, b, pos, m.v).double()
            for h in range(heads):
                j, q = h // group, m.q[b, h].double()
                x = scale * (k[:, j] @ q)
                lse[h] = torch.logsumexp(x, 0)
                p = torch.exp(x - lse[h])
                out[h] = p @ v[:, j]
                # A logit is a 32-bit sum of dim products and a few roundings of
                # it (the scale, base 2, the difference to the maximum).
                ex = ((m.dim + 4) * F32 * abs(scale) * (k[:, j].abs() @ q.abs()) + 6 * F32 * x.abs()).max()
                ex = ex + 6 * F32 * (x.max() - x.min())
                # A weight: the exponential of two such logits' difference, its
                # own rounding (2 units of 32 bits), and 32-bit sums.  A run of n
                # terms is summed in partial sums no longer than n / 64 + 64.
                sums = (n / 64 + 64) * F32
                ep = 2 * ex + 4 * F32 + 2 * sums
                lse_tol[h] = ex + 4 * F32 + sums + 2 * F32 * lse[h].abs()
                w[j, pos] += p
                w_tol[j, pos] += (ep + (group + 2) * F32) * p
                mix = p @ v[:, j].abs()
                out_tol[h] = UNIT[m.dtype] * out[h].abs() + (ep + WEIGHT[m.dtype]) * mix * (1 + UNIT[m.dtype])
                # subnormal results of the 16-bit type round to its smallest step
                out_tol[h] += torch.finfo(m.dtype).smallest_normal * torch.finfo(m.dtype).eps
        res.append((out, out_tol, lse, lse_tol, w, w_tol))
    return res


def key(x):
    """Order of masses: NaN above all."""
    return (1, 0.0) if math.isnan(x) else (0, x)


def evict(mass, n, budget, sinks, recent):
    """Kept positions of one KV head."""
    if n <= budget:
        return list(range(n))
    mid = sorted(range(sinks, n - recent), key=lambda t: (tuple(-v for v in key(float(mass[t]))), t))
    mid = sorted(mid[:budget - sinks - recent])
    return list(range(sinks)) + mid + list(range(n - recent, n))
