"""The cache as a serving program uses it, two layers: a prompt is cached, its
sequence forked, the samples grow token by token with attention behind the
common prompt, beams are chosen, sequences end, the pool is compacted, a
sequence leaves through the codec and returns.  Everything is compared with
plain lists of every sequence's rows."""
import random

import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
import kv_shared_reference as H
from test_gpu_kv_pages import Made, ints
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu
KVH, DIM, PAGE, HEADS, LAYERS = 2, 64, 16, 24, 2


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Program:
    def __init__(self, batch, pages, width, seed):
        self.batch, self.rng = batch, random.Random(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.kv = torch.zeros(LAYERS, 2, pages, KVH, PAGE, DIM, dtype=torch.bfloat16, device=DEV)
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.caches = [S.KVCache(k, v, self.table, self.lens) for k, v in self.kv]
        self.pages = S.KVPages(self.caches)
        self.pages.count()
        self.ws = S.KVSharedWorkspace(self.caches[0], HEADS)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.rows = [torch.zeros(0, LAYERS, 2, KVH, DIM, dtype=torch.bfloat16) for _ in range(batch)]      # what is cached

    def grow(self, more):
        """more[b] new tokens of every sequence, in all layers."""
        lens = [len(r) + n for r, n in zip(self.rows, more)]
        self.pages.resize(ints(lens), status=self.status)
        new = [torch.randn(n, LAYERS, 2, KVH, DIM, generator=self.gen).to(torch.bfloat16) for n in more]
        cu = ints([sum(more[:b]) for b in range(self.batch + 1)])
        flat = torch.cat(new).to(DEV)
        for i, c in enumerate(self.caches):
            c.append(flat[:, i, 0], flat[:, i, 1], cu, status=self.status)
        self.rows = [torch.cat([r, x]) for r, x in zip(self.rows, new)]

    def fork(self, parents):
        self.pages.fork(ints(parents), status=self.status)
        self.rows = [self.rows[p] if p >= 0 else self.rows[0][:0] for p in parents]

    def cut(self, lens):
        self.pages.resize(ints(lens), status=self.status)
        self.rows = [r[:n] for r, n in zip(self.rows, lens)]

    def check(self, what):
        torch.cuda.synchronize()
        assert int(self.status) == 0, what
        assert self.lens.tolist() == [len(r) for r in self.rows], what
        table, kv = self.table.cpu(), self.kv.cpu()
        named = torch.bincount(table[table >= 0].long(), minlength=kv.shape[2])
        assert self.pages.refs.tolist() == named.tolist(), what
        for b, r in enumerate(self.rows):
            t = torch.arange(len(r))
            where, slot = table[b].long()[t // PAGE], t % PAGE
            got = kv[:, :, where, :, slot]                      # [token, layers, 2, kv_heads, dim]
            assert torch.equal(got.view(torch.int16), r.view(torch.int16)), (what, b)

    def attend(self, cu, shared, what):
        q = torch.randn(self.batch, HEADS, DIM, generator=self.gen).to(torch.bfloat16)
        for i, c in enumerate(self.caches):
            lse = torch.zeros(self.batch, HEADS, device=DEV)
            out = c.attend_shared(q.to(DEV), ints(cu), ints(shared), self.ws, lse=lse, status=self.status)
            m = R.Made()
            m.lens, m.kv_heads, m.dim, m.page, m.dtype = [len(r) for r in self.rows], KVH, DIM, PAGE, torch.bfloat16
            m.table, m.q, m.cu, m.shared = self.table.cpu(), q, cu, shared
            m.k, m.v = self.kv[i].cpu()
            for b, (o, o_tol, e, e_tol) in enumerate(H.attend(m)):
                assert bool(((out[b].double().cpu() - o).abs() <= o_tol).all()), (what, i, b)
                if m.lens[b]:
                    assert bool(((lse[b].double().cpu() - e).abs() <= e_tol).all()), (what, i, b)


@pytest.mark.parametrize("width", [40, 3000])
def test_a_serving_program(width):
    """A table of its sequences' size, and one so wide that the other attention kernel is chosen."""
    _say("a serving program, table for %d pages" % width)
    p = Program(7, 200, width, seed=3)
    prompt = 300
    p.grow([prompt, 0, 0, 0, 0, 45, 0])
    p.check("prompts")
    p.fork([0, 0, 0, 0, 0, 5, 6])                    # five samples of the first prompt
    p.check("samples")
    cu, shared = [0, 5, 6, 7], [prompt, 0, 0]
    for step in range(3):
        p.grow([1, 1, 1, 1, 1, 1, 0])
        p.attend(cu, shared, step)
    p.check("steps")
    p.fork([2, 2, 0, 4, 4, 5, -1])                   # beams are chosen
    p.grow([1] * 5 + [20, 0])
    p.check("beams")
    p.attend(cu, shared, "beams")
    p.grow([8, 8, 8, 8, 8, 0, 0])                    # drafts ...
    p.cut([prompt + 4 + n for n in (0, 3, 8, 1, 0)] + [len(p.rows[5]), 0])      # ... and what was taken of them
    p.check("drafts")
    p.attend(cu, shared, "drafts")
    p.fork([0, -1, 2, -1, 4, 5, 6])                  # two end
    used = p.pages.compact(status=p.status)
    p.check("compacted")
    held = int((p.table >= 0).sum())
    assert int(used) == len(set(p.table[p.table >= 0].tolist())) <= held
    assert int(p.table.max()) == int(used) - 1
    p.attend(cu, shared, "compacted")
    # a sequence leaves, its pages are given back, and it returns in another's place
    ws = S.Workspace(KVH * 400 * DIM, device=DEV)
    packed = [S.persist.pack_sequence("layer.%d" % i, c, 2, ws) for i, c in enumerate(p.caches)]
    kept = p.rows[2]
    p.fork([0, 1, -1, 3, 4, 5, 6])
    p.check("left")
    lens = [len(r) for r in p.rows]
    lens[3] = len(kept)
    p.pages.resize(ints(lens), status=p.status)
    for c, x in zip(p.caches, packed):
        assert S.persist.unpack_sequence(x, c, 3) == len(kept)
    p.rows[3] = kept
    p.check("returned")
    p.attend(cu, shared, "returned")
    p.fork([-1] * 7)
    p.check("over")
    assert int(p.pages.refs.sum()) == 0 and int(p.pages.compact()) == 0


def test_steps_of_two_programs_captured_and_on_streams():
    """Fork, resize and compact of two pools on streams of their own, and captured in two graphs that are replayed
    together, with other parents and lengths every time."""
    _say("page operators on two streams, in two graphs")
    made = [Made([40, 3, 17, 0], 90, 8, 12, layers=2, kv_heads=2, dim=16, seed=s, layout=l) for s, l in ((1, "hnd"), (2, "nhd"))]
    arg = [(ints([0, 1, 2, 3]), ints([40, 3, 17, 0])) for _ in made]
    streams = [torch.cuda.Stream() for _ in made]
    for m in made:
        m.count()

    def step(m, a, stream=None):
        how = dict(status=m.status, stream=stream)
        m.pages.fork(a[0], **how)
        m.pages.resize(a[1], **how)
        m.pages.compact(moved=m.moved, used=m.used, **how)

    graphs = []
    for m, a in zip(made, arg):
        m.used = torch.zeros(1, dtype=torch.int32, device=DEV)
        step(m, a)
        m.ref.resize([40, 3, 17, 0])
        m.ref.compact()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(m, a)
        graphs.append(g)
    rng = random.Random(5)
    for rep in range(8):
        want = []
        for m, a in zip(made, arg):
            parents = [rng.choice([b, rng.randrange(4), -1]) for b in range(4)]
            m.ref.fork(parents)
            lens = [min(96, max(0, n + rng.choice([-9, 1, 1, 20]))) for n in m.ref.lens]
            m.ref.resize(lens)
            want.append(m.ref.compact())
            a[0].copy_(ints(parents))
            a[1].copy_(ints(lens))
        torch.cuda.synchronize()
        for m, a, g, stream in zip(made, arg, graphs, streams):
            if rep % 2:
                step(m, a, stream)
            else:
                with torch.cuda.stream(stream):
                    g.replay()
        torch.cuda.synchronize()
        for m, (used, moved) in zip(made, want):
            m.check(rep)
            assert int(m.used) == used and m.moved.tolist() == moved


def test_a_whole_step_captured():
    """Room for a token, its append and the attention in one graph, replayed; checked against the plain lists."""
    _say("a step in a graph")
    p = Program(4, 60, 12, seed=9)
    p.grow([90, 0, 0, 30])
    p.fork([0, 0, 0, 3])
    one, cu = torch.ones(4, dtype=torch.int32, device=DEV), ints([0, 1, 2, 3, 4])
    groups, shared = ints([0, 3, 4]), ints([90, 0])
    new = torch.zeros(4, LAYERS, 2, KVH, DIM, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(4, HEADS, DIM, dtype=torch.bfloat16, device=DEV)
    out = [torch.zeros_like(q) for _ in p.caches]
    target = torch.zeros(4, dtype=torch.int32, device=DEV)

    def step():
        torch.add(p.lens, one, out=target)
        p.pages.resize(target, status=p.status)
        for i, c in enumerate(p.caches):
            c.append(new[:, i, 0], new[:, i, 1], cu, status=p.status)
            c.attend_shared(q, groups, shared, p.ws, out=out[i], status=p.status)

    def fill():
        new.copy_(torch.randn(new.shape, generator=p.gen))
        q.copy_(torch.randn(q.shape, generator=p.gen))
        p.rows = [torch.cat([r, x[None]]) for r, x in zip(p.rows, new.cpu())]

    fill()
    step()
    p.check("eager")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(20):
        fill()
        g.replay()
        p.check(rep)
        for i, c in enumerate(p.caches):
            want = c.attend_shared(q, groups, shared, p.ws)
            assert torch.equal(out[i].view(torch.int16), want.view(torch.int16)), rep
    p.attend([0, 3, 4], [90, 0], "at the end")
