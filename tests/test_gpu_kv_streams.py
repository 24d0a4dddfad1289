"""Append, gather and eviction on streams of their own, two caches at once, and
captured together: a step that appends, attends, evicts into other pages and
gathers what stays."""
import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view(torch.int16)


class Step:
    """A cache, a destination for its eviction, and the step's tensors."""

    def __init__(self, seed, lens=(300, 1, 90, 0), budget=64):
        self.lens, self.budget, n = list(lens), budget, len(lens)
        self.m = R.to_gpu(R.make(lens, 2, 64, 16, torch.bfloat16, heads=4, seed=seed, fill=0.0), S)
        self.to = R.to_gpu(R.make([min(x, budget) for x in lens], 2, 64, 16, torch.bfloat16, seed=seed + 50, fill=0.0), S)
        self.ws = S.KVWorkspace(self.m.cache, 4, mass=True)
        has = [min(x, 1) for x in lens]
        self.cu = torch.tensor([sum(has[:b]) for b in range(n + 1)], dtype=torch.int32, device=DEV)
        kept = [min(x, budget) for x in lens]
        self.cu_kept = torch.tensor([sum(kept[:b]) for b in range(n + 1)], dtype=torch.int32, device=DEV)
        self.k, self.v = (torch.zeros(sum(has), 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.back = [torch.zeros(sum(kept), 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        self.mass = torch.zeros(n, 2, max(lens), device=DEV)
        self.mass_to = torch.zeros_like(self.mass)
        self.out = torch.zeros_like(self.m.gq)
        self.kept = torch.zeros(n, 2, budget, dtype=torch.int32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        for t in (self.k, self.v, self.m.gq):
            t.copy_(torch.randn(t.shape, generator=g))
        self.mass.copy_(torch.rand(self.mass.shape, generator=g))
        for t in (*self.back, self.mass_to, self.out, self.to.gk, self.to.gv):
            t.zero_()

    def run(self, stream=None):
        how = dict(status=self.status, stream=stream)
        self.m.cache.append(self.k, self.v, self.cu, **how)
        self.m.cache.attend(self.m.gq, self.ws, out=self.out, mass=self.mass, **how)
        self.m.cache.evict(self.mass, self.budget, sinks=2, recent=8, to=self.to.cache, kept=self.kept,
                           mass_out=self.mass_to, **how)
        self.to.cache.gather(*self.back, self.cu_kept, **how)

    def check(self):
        """Against the plain eviction of the mass that the attention left."""
        assert int(self.status) == 0
        mass, new_k, new_v = self.mass.cpu(), self.m.gk.cpu(), self.m.gv.cpu()
        at = 0
        for b, n in enumerate(self.lens):
            size = min(n, self.budget)
            assert int(self.to.glens[b]) == size
            for h in range(2):
                keep = R.evict(mass[b, h], n, self.budget, 2, 8)
                assert self.kept[b, h, :size].tolist() == keep
                for back, pool in zip(self.back, (new_k, new_v)):
                    assert torch.equal(bits(back[at:at + size, h].cpu()), bits(R.rows(self.m, b, keep, pool)[:, h]))
            if n:       # the step's token is in its place
                row = int(self.cu[b])
                assert torch.equal(bits(R.rows(self.m, b, [n - 1], new_k)[0]), bits(self.k[row].cpu()))
            at += size

    def results(self):
        return [t.clone() for t in (self.out, self.mass, self.kept, self.mass_to, *self.back)]


def test_two_caches_on_streams_of_their_own():
    _say("append, attend, evict and gather on two streams")
    steps = [Step(1), Step(2, (40, 500, 2, 65, 64))]
    streams = [torch.cuda.Stream() for _ in steps]
    for rep in range(4):
        want = []
        for i, s in enumerate(steps):
            s.fill(10 * rep + i)
            s.run()
            want.append(s.results())
            s.fill(10 * rep + i)
        torch.cuda.synchronize()
        for s, stream in zip(steps, streams):
            s.run(stream)
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            s.check()
            for got, t in zip(s.results(), w):
                assert torch.equal(got.view(torch.uint8), t.view(torch.uint8)), rep


def test_a_step_captured_and_replayed():
    _say("append, attend, evict and gather in a graph")
    s = Step(3)
    s.fill(0)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for rep in range(6):
        s.fill(rep)
        s.run()
        want = s.results()
        s.fill(rep)
        g.replay()
        torch.cuda.synchronize()
        s.check()
        for got, t in zip(s.results(), want):
            assert torch.equal(got.view(torch.uint8), t.view(torch.uint8)), rep
