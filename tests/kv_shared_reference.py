"""Caches whose sequences begin alike, and a 64-bit reference of attention over
them with error bounds.  No code of the package."""
import math

import torch

import kv_reference as R
from kv_reference import F32, UNIT, WEIGHT


def make(groups, kv_heads, dim, page, dtype, heads, layout="hnd", seed=0, width=None, fill=float("nan"), k_scale=1.0):
    """``groups``: (tokens in common, [lengths]) each.  The pages that the
    tokens in common fill are in all members' rows; the one that they begin is
    every member's own, with the same values."""
    lens = [n for _, members in groups for n in members]
    m = R.make(lens, kv_heads, dim, page, dtype, layout=layout, seed=seed, heads=heads, width=width, fill=fill, k_scale=k_scale)
    m.cu, m.shared, b = [0], [c for c, _ in groups], 0
    for common, members in groups:
        first = b
        for n in members:
            c = min(common, lens[first], n)
            full = c // page
            if b > first and c:
                if c % page:
                    for pool in (m.k, m.v):
                        pool[int(m.table[b, full]), :, :c % page] = pool[int(m.table[first, full]), :, :c % page]
                m.table[b, :full] = m.table[first, :full]
            b += 1
        m.cu.append(b)
    return m


def common_of(m):
    """Per sequence the tokens that are attended for its group."""
    out = [0] * len(m.lens)
    for g, common in enumerate(m.shared):
        lo, hi = m.cu[g], m.cu[g + 1]
        if 0 <= lo <= hi <= len(m.lens) and hi - lo > 1:
            c = min(max(common, 0), m.lens[lo])
            for b in range(lo, hi):
                out[b] = c if m.lens[b] >= c else 0
    return out


def attend(m, scale=None, hidden=()):
    """Per sequence: out [heads, dim], lse [heads] and bounds of their errors.
    ``hidden``: (sequence, position) left out."""
    scale = m.dim ** -0.5 if scale is None else scale
    heads = m.q.shape[1]
    group, unit, common = heads // m.kv_heads, UNIT[m.dtype], common_of(m)
    res = []
    for b, n in enumerate(m.lens):
        out, out_tol = torch.zeros(heads, m.dim, dtype=torch.float64), torch.zeros(heads, m.dim, dtype=torch.float64)
        lse, lse_tol = torch.full((heads,), -math.inf, dtype=torch.float64), torch.zeros(heads, dtype=torch.float64)
        pos = [t for t in range(n) if (b, t) not in hidden]
        if pos:
            k, v = R.rows(m, b, pos, m.k).double(), R.rows(m, b, pos, m.v).double()
            before = torch.tensor([t < common[b] for t in pos])
            for h in range(heads):
                j, q = h // group, m.q[b, h].double()
                x = scale * (k[:, j] @ q)
                lse[h] = torch.logsumexp(x, 0)
                p = torch.exp(x - lse[h])
                out[h] = p @ v[:, j]
                # Logits and weights as in kv_reference.  A lane adds up two of 8 tokens at a time, where one
                # workgroup has all tokens in common n / 8 times.
                ex = ((m.dim + 4) * F32 * abs(scale) * (k[:, j].abs() @ q.abs()) + 6 * F32 * x.abs()).max()
                ex = ex + 6 * F32 * (x.max() - x.min())
                sums = (n / 8 + 64) * F32
                ep = 2 * ex + 4 * F32 + 2 * sums
                lse_tol[h] = ex + 4 * F32 + sums + 2 * F32 * lse[h].abs()
                # The weights of tokens in common are rounded to the type, half a step each; in fp16, where they are
                # held times 2^11, no weight is held below the step 2^-24, which adds 2^-35 of the largest (at most 1).
                mix = p @ v[:, j].abs()
                rounded = unit * (p * before) @ v[:, j].abs()
                if m.dtype is torch.float16:
                    rounded = rounded + 2.0 ** -35 * v[before, j].abs().sum(0)
                out_tol[h] = unit * out[h].abs() + ((ep + WEIGHT[m.dtype]) * mix + rounded) * (1 + unit) ** 2
                out_tol[h] += torch.finfo(m.dtype).smallest_normal * torch.finfo(m.dtype).eps
        res.append((out, out_tol, lse, lse_tol))
    return res
