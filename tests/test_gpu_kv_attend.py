"""Attention of one new token over a paged cache, with windows, sinks and the
accumulated weights, against a 64-bit reference."""
import math

import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(m, window=None, sinks=0, scale=None, want_mass=True, hidden=(), want_status=0):
    heads = m.q.shape[1]
    ws = S.KVWorkspace(m.cache, heads, mass=want_mass)
    ws.buf.fill_(0xA5)
    lse = torch.full((len(m.lens), heads), 7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(m.gq, 5.0)
    width = max(m.lens + [1]) + 3
    mass = torch.rand(len(m.lens), m.kv_heads, width, device=DEV) if want_mass else None
    before = mass.cpu() if want_mass else None
    m.cache.attend(m.gq, ws, out=out, window=window, sinks=sinks, scale=scale, lse=lse, mass=mass, status=status)
    if want_mass:
        mass_out = torch.full_like(mass, -3.0)
        out2 = m.cache.attend(m.gq, ws, window=window, sinks=sinks, scale=scale, mass=before.to(DEV),
                              mass_out=mass_out)
        assert torch.equal(out2.view(torch.int16), out.view(torch.int16))
    else:
        out2 = m.cache.attend(m.gq, ws, window=window, sinks=sinks, scale=scale)
        assert torch.equal(out2.view(torch.int16), out.view(torch.int16))
    torch.cuda.synchronize()
    assert int(status.item()) == want_status
    for b, (o, o_tol, e, e_tol, w, w_tol) in enumerate(R.attend(m, scale, window, sinks, hidden)):
        n = m.lens[b]
        got = out[b].double().cpu()
        assert bool(((got - o).abs() <= o_tol).all()), (b, float(((got - o).abs() - o_tol).max()))
        seen = ~torch.isinf(e)
        le = lse[b].double().cpu()
        assert torch.equal(torch.isinf(le), ~seen), b
        assert bool((le[~seen] < 0).all())
        assert bool(((le[seen] - e[seen]).abs() <= e_tol[seen]).all()), (b, (le[seen] - e[seen]).abs().max(), e_tol)
        if want_mass:
            sums = before[b, :, :n].double() + w
            tol = w_tol + R.F32 * sums.abs()
            for got_mass in (mass, mass_out):
                gm = got_mass[b, :, :n].double().cpu()
                assert bool(((gm - sums).abs() <= tol).all()), (b, float(((gm - sums).abs() - tol).max()))
            assert torch.equal(mass[b, :, n:].cpu(), before[b, :, n:])
            assert bool((mass_out[b, :, n:] == -3.0).all())
    return out


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [8, 64, 72, 80, 96, 128, 192, 200, 256])
@pytest.mark.parametrize("group", [1, 5])
def test_dims(dtype, dim, group):
    _say("attend dim=%d group=%d %s" % (dim, group, dtype))
    m = R.make([0, 1, 2, 31, 33, 300], 2, dim, 16, dtype, heads=2 * group, seed=dim + group)
    check(R.to_gpu(m, S))


@pytest.mark.parametrize("group", [1, 2, 3, 8, 15, 16, 17, 32, 33, 48, 64, 65, 130])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_groups(group, dim):
    _say("attend group=%d dim=%d" % (group, dim))
    m = R.make([77, 1, 0, 515], 2, dim, 32, BF16, layout="nhd", heads=2 * group, seed=group)
    check(R.to_gpu(m, S))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,group", [(40, 20), (24, 64), (72, 24), (104, 64), (168, 20), (176, 48), (208, 24), (248, 32)])
def test_odd_dims_of_many_rows(dim, group, dtype):
    """Head sizes between the kernels' own with several blocks of query rows,
    whole and cut into runs."""
    _say("attend dim=%d group=%d %s" % (dim, group, dtype))
    for width in (None, 500):
        m = R.make([40, 0, 333, 129, 1], 2, dim, 16, dtype, heads=2 * group, seed=dim, width=width)
        check(R.to_gpu(m, S))


@pytest.mark.parametrize("page", [1, 2, 7, 8, 16, 24, 33, 64, 128, 1000])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_pages(page, layout):
    _say("attend page=%d %s" % (page, layout))
    lens = [0, 1, page - 1, page, page + 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500]
    m = R.make(lens, 3, 128, page, FP16 if page % 2 else BF16, layout=layout, heads=12, seed=page)
    check(R.to_gpu(m, S))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,group", [(8, 3), (64, 1), (64, 20), (64, 50), (80, 4), (80, 64), (128, 1), (128, 16),
                                       (128, 31), (128, 33), (128, 64), (128, 70), (192, 2), (192, 32), (256, 1),
                                       (256, 17), (256, 40)])
def test_tables_far_wider_than_the_sequences(dim, group, dtype):
    """A serving loop's table: what it could hold decides how the work is cut,
    what it holds is short, ragged or nothing."""
    _say("attend wide table dim=%d group=%d %s" % (dim, group, dtype))
    m = R.make([0, 1, 300, 31, 0, 700, 129, 2], 2, dim, 16, dtype, layout="nhd", heads=2 * group, seed=group, width=600)
    check(R.to_gpu(m, S))
    check(m, window=200, sinks=5, want_mass=False)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 4), (1, 0), (1, 1), (16, 4), (100, 0), (100, 33), (128, 64),
                                          (511, 1), (512, 4), (2 ** 31 - 1, 5), (7, 2 ** 31 - 1), (None, 9)])
def test_windows(window, sinks):
    _say("attend window=%s sinks=%d" % (window, sinks))
    m = R.make([0, 1, 5, 16, 40, 129, 512, 513, 700], 2, 64, 16, BF16, heads=8, seed=3)
    check(R.to_gpu(m, S), window=window, sinks=sinks)


@pytest.mark.parametrize("lens", [[5000], [4096, 1], [1] * 70, [0] * 5, [9000, 0, 0, 3, 2000], list(range(130))])
@pytest.mark.parametrize("want_mass", [False, True])
def test_batches(lens, want_mass):
    _say("attend %d sequences up to %d mass=%s" % (len(lens), max(lens), want_mass))
    m = R.make(lens, 1 if len(lens) == 130 else 2, 64, 16, BF16, heads=4, seed=len(lens))
    check(R.to_gpu(m, S), want_mass=want_mass)


@pytest.mark.parametrize("batch", [64, 65, 150, 400])
def test_many_sequences_cut_into_runs(batch):
    """More sequences than a wave has lanes, none of them whole in a run."""
    _say("attend %d sequences in a wide table" % batch)
    lens = [(37 * b) % 301 if b % 7 else 0 for b in range(batch)]
    lens[-1] = 700
    m = R.make(lens, 1, 64, 16, BF16, heads=3, seed=batch, width=64)
    check(R.to_gpu(m, S))
    check(m, window=64, sinks=4, want_mass=False)


def test_sequences_beyond_a_wave_of_blocks():
    """More than 64 times 64 of them: their blocks' sums take a second look."""
    lens = [(13 * b) % 40 if b % 5 else 0 for b in range(4200)]
    lens[0], lens[4101], lens[-1] = 900, 500, 300
    _say("attend %d sequences" % len(lens))
    check(R.to_gpu(R.make(lens, 1, 64, 16, BF16, heads=2, seed=3, width=64), S))


def test_output_in_place_of_the_queries():
    m = R.to_gpu(R.make([2000, 0, 33], 2, 128, 16, BF16, heads=8, seed=6), S)
    ws = S.KVWorkspace(m.cache, 8)
    want = m.cache.attend(m.gq, ws)
    assert m.cache.attend(m.gq, ws, out=m.gq) is m.gq
    assert torch.equal(m.gq.view(torch.int16), want.view(torch.int16))


def test_peaked_and_far_logits():
    """Logits in the hundreds: one token takes all, whatever tile it is in; and
    a maximum that grows from tile to tile."""
    m = R.make([700, 3], 1, 128, 16, BF16, heads=4, seed=8)
    m.k[m.table[0, 20].long(), 0, 3] = m.q[0, 0] * 40
    check(R.to_gpu(m, S), scale=0.7)
    m = R.make([900], 1, 64, 16, FP16, heads=1, seed=9)
    t = torch.arange(900)
    m.q[:] = 1.0
    m.k[m.table[0].long()[t // 16], 0, t % 16] = (t[:, None].float() / 64).to(FP16).expand(900, 64).clone()
    check(R.to_gpu(m, S))
    check(m, scale=-1.0)
    check(m, scale=0.0)


def test_many_small_weights_in_fp16():
    """One heavy token and thousands 12 to 16 nats below it: their weights are
    small numbers of the type, and must still add up."""
    n = 6000
    m = R.make([n], 1, 64, 64, FP16, heads=2, seed=10)
    t = torch.arange(n)
    m.q[:] = 0.25
    depth = torch.where(t == 17, torch.zeros(n), -12.0 - 4.0 * (t % 5) / 4)
    m.k[m.table[0].long()[t // 64], 0, t % 64] = (depth / (64 * 0.25 * 0.125))[:, None].to(FP16).expand(n, 64).clone()
    m.v[m.table[0].long()[t // 64], 0, t % 64] = 1.0 + (t[:, None] % 7).to(FP16).expand(n, 64).clone() / 8
    m.v[m.table[0, 0].long(), 0, 17] = 0
    check(R.to_gpu(m, S))


def test_lowest_and_infinite_values():
    """The type's lowest value and infinities in K: a logit of -inf or of the
    lowest value weighs nothing beside an ordinary one; infinite V under a
    visible token comes through; under hidden tokens nothing does."""
    for dtype in (BF16, FP16):
        m = R.make([200], 1, 64, 16, dtype, heads=1, seed=4, fill=math.inf)
        m.q[:] = 0.0
        m.q[0, 0, 0] = 1.0
        low = torch.finfo(dtype).min
        for t, x in ((3, low), (50, -math.inf), (150, low)):
            m.k[m.table[0, t // 16].long(), 0, t % 16, 0] = x
        R.to_gpu(m, S)
        ws = S.KVWorkspace(m.cache, 1)
        out = m.cache.attend(m.gq, ws)
        # the same without those tokens
        r = R.attend(m, hidden={(0, 3), (0, 50), (0, 150)})[0]
        assert bool(((out[0].double().cpu() - r[0]).abs() <= r[1]).all())
        m.v[m.table[0, 0].long(), 0, 5, 7] = math.inf
        m.gv.copy_(m.v)
        out = m.cache.attend(m.gq, ws)
        assert out[0, 0, 7].item() == math.inf and bool(torch.isfinite(out[0, 0, :7]).all())
        # outside the window it is not seen, nor is a NaN
        m.v[m.table[0, 0].long(), 0, 6, 8] = math.nan
        m.k[m.table[0, 0].long(), 0, 7, 0] = math.nan
        m.gv.copy_(m.v)
        m.gk.copy_(m.k)
        out = m.cache.attend(m.gq, ws, window=100, sinks=3)
        r = R.attend(m, window=100, sinks=3, hidden={(0, 150)})[0]
        assert bool(((out[0].double().cpu() - r[0]).abs() <= r[1]).all())
        # visible, a NaN logit makes the row NaN, as the formula does
        assert bool(torch.isnan(m.cache.attend(m.gq, ws)).all())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,heads", [(64, 1), (128, 20), (72, 3), (256, 2)])
def test_infinite_v_whatever_its_weight(dim, heads, dtype):
    """Infinities in V under tokens of every weight, the largest (exactly 1
    before the division) among them: infinite in their columns and of their
    sign, all others as without them."""
    n = 160
    m = R.make([n], 1, dim, 16, dtype, heads=heads, seed=12)
    R.to_gpu(m, S)
    ws = S.KVWorkspace(m.cache, heads)
    want = R.attend(m)[0]
    top = int((m.k[m.table[0].long()].float().permute(0, 2, 1, 3).reshape(-1, dim)[:n] @ m.q[0, 0].float()).argmax())
    for step, tokens in enumerate([[top]] + [range(i, n, 40) for i in range(40)]):
        v = m.v.clone()
        cols = torch.zeros(dim, dtype=torch.float64)
        for i, t in enumerate(tokens):
            col = (5 * step + 13 * i) % dim
            x = math.inf if i % 2 == 0 else -math.inf
            if cols[col]:
                continue
            v[m.table[0, t // 16].long(), 0, t % 16, col] = x
            cols[col] = x
        m.gv.copy_(v)
        out = m.cache.attend(m.gq, ws)[0].double().cpu()
        hit = cols != 0
        assert torch.equal(out[:, hit], cols[hit].expand(heads, -1)), step
        assert bool(((out - want[0]).abs() <= want[1])[:, ~hit].all()), step


@pytest.mark.parametrize("dtype,size,scale", [(BF16, 1e-39, 1e34), (BF16, 3e-38, 1e34), (FP16, 1e-6, 125.0),
                                              (FP16, 6e-8, 2000.0)])
def test_subnormal_values(dtype, size, scale):
    """Subnormal K and V count for what they are."""
    m = R.make([200, 3], 1, 64, 16, dtype, heads=4, seed=1, fill=0.0)
    m.v = (torch.randn(m.v.shape, generator=torch.Generator().manual_seed(2)) * size).to(dtype)
    check(R.to_gpu(m, S))
    m = R.make([200, 3], 1, 64, 16, dtype, heads=4, seed=1, fill=0.0)
    m.k = (m.k.float() * size).to(dtype)
    m.q = (m.q.float() * 1000).to(dtype)
    check(R.to_gpu(m, S), scale=scale)


def test_every_logit_minus_infinity_gives_zeros():
    m = R.make([40, 5], 1, 64, 16, BF16, heads=2, seed=4)
    m.q[:] = 1.0
    m.k[m.table[0].long()[:3]] = -math.inf
    R.to_gpu(m, S)
    lse = torch.zeros(2, 2, device=DEV)
    mass = torch.ones(2, 1, 40, device=DEV)
    out = m.cache.attend(m.gq, S.KVWorkspace(m.cache, 2, mass=True), lse=lse, mass=mass)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all()) and bool((mass[0] == 1).all())
    assert bool(torch.isfinite(out[1].float()).all()) and bool((out[1] != 0).any())


def test_strided_tensors():
    """Queries and outputs inside larger ones, pools that share one
    allocation, a mass and a table with rows apart, an odd mass stride."""
    m = R.make([90, 0, 33], 2, 128, 16, BF16, heads=4, seed=6)
    both = torch.full((m.k.shape[0], 2, 2, 16, 128), math.nan, dtype=BF16, device=DEV)
    both[:, 0], both[:, 1] = m.k.to(DEV), m.v.to(DEV)
    table = torch.full((3, m.table.shape[1] + 5), 1 << 30, dtype=torch.int32, device=DEV)
    table[:, :m.table.shape[1]] = m.table.to(DEV)
    R.to_gpu(m, S)
    m.cache = S.KVCache(both[:, 0], both[:, 1], table[:, :m.table.shape[1]], m.glens)
    packed = torch.randn(3, 4 + 2 + 2, 128, device=DEV).to(BF16)
    packed[:, :4] = m.gq
    m.gq = packed[:, :4]
    ref = R.attend(m)
    wide = torch.full((4, 3, 160), 9.0, dtype=BF16, device=DEV)
    out = wide.transpose(0, 1)[:, :, 16:144]
    mass = torch.zeros(3, 3, 95, device=DEV)
    m.cache.attend(m.gq, S.KVWorkspace(m.cache, 4, mass=True), out=out, mass=mass[:, 1:, 1:92])
    for b in range(3):
        assert bool(((out[b].double().cpu() - ref[b][0]).abs() <= ref[b][1]).all())
        n = m.lens[b]
        assert bool(((mass[b, 1:, 1:n + 1].double().cpu() - ref[b][4]).abs() <= ref[b][5]).all())
    assert bool((mass[:, 0] == 0).all()) and bool((mass[:, :, 0] == 0).all()) and bool((wide[:, :, :16] == 9).all())
    assert bool((wide[:, :, 144:] == 9).all())


def test_bad_pages_and_lengths():
    """A page number outside the pool hides its tokens; a length outside the
    table is cut; both are reported."""
    m = R.make([100, 64, 10], 2, 64, 16, BF16, heads=4, seed=12, width=7)
    hidden = {(0, t) for t in range(16, 32)} | {(1, t) for t in range(48, 64)}
    good = m.table.clone()
    m.table[0, 1], m.table[1, 3] = -1, m.k.shape[0]
    R.to_gpu(m, S)
    m.table = good
    check(m, hidden=hidden, want_status=1)
    m.gtable.copy_(good)
    m.glens[0], m.glens[2] = 7 * 16 + 1, -4
    m.gtable[0] = torch.arange(7, dtype=torch.int32, device=DEV) % m.k.shape[0]
    m.table[0], m.lens = m.gtable[0].cpu(), [112, 64, 0]
    m.gk.copy_(torch.nan_to_num(m.gk))
    m.gv.copy_(torch.nan_to_num(m.gv))
    m.k, m.v = m.gk.cpu(), m.gv.cpu()
    check(m, want_status=2)


def test_mass_shorter_than_the_sequence():
    m = R.to_gpu(R.make([50], 1, 64, 16, BF16, heads=2, seed=13), S)
    mass = torch.zeros(1, 1, 64, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.cache.attend(m.gq, S.KVWorkspace(m.cache, 2, mass=True), mass=mass[:, :, :20], status=status)
    w, tol = R.attend(m)[0][4:]
    assert int(status) == 2
    assert bool(((mass[0, :, :20].double().cpu() - w[:, :20]).abs() <= tol[:, :20]).all())
    assert bool((mass[0, :, 20:] == 0).all())


def test_offsets_past_32_bits():
    """Pages far apart: byte offsets pass 2^32 and element offsets 2^31."""
    lens, dim, page = [70], 64, 16
    m = R.make(lens, 1, dim, page, BF16, heads=3, seed=14, slack=0)
    far = (1 << 30) + 8          # elements between pages: 5 pages span 8 GiB
    buf = torch.empty(far * 4 + page * dim, dtype=BF16, device=DEV)
    pool = buf.as_strided((5, 1, page, dim), (far, page * dim, dim, 1))
    R.to_gpu(m, S)
    pool.copy_(m.gk)
    m.cache = S.KVCache(pool, m.gv, m.gtable, m.glens)
    check(m)
    m.cache = S.KVCache(m.gk, pool.copy_(m.gv), m.gtable, m.glens)
    check(m)


def test_other_stream_and_two_at_once():
    ms = [R.to_gpu(R.make([3000, 17], 2, 128, 16, BF16, heads=8, seed=20 + i), S) for i in range(2)]
    refs = []
    for m in ms:
        refs.append(m.cache.attend(m.gq, S.KVWorkspace(m.cache, 8)).clone())
    streams = [torch.cuda.Stream() for _ in ms]
    wss = [S.KVWorkspace(m.cache, 8) for m in ms]
    torch.cuda.synchronize()
    for rep in range(4):
        outs = [m.cache.attend(m.gq, ws, stream=st) for m, ws, st in zip(ms, wss, streams)]
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            assert torch.equal(o.view(torch.int16), r.view(torch.int16)), rep


def test_repeats_are_bit_equal():
    m = R.to_gpu(R.make([9000, 300, 0, 41], 2, 128, 16, BF16, heads=16, seed=30), S)
    ws = S.KVWorkspace(m.cache, 16, mass=True)
    runs = []
    for _ in range(5):
        mass = torch.zeros(4, 2, 9000, device=DEV)
        runs.append((m.cache.attend(m.gq, ws, mass=mass).clone(), mass))
    for o, ms in runs[1:]:
        assert torch.equal(o.view(torch.int16), runs[0][0].view(torch.int16)) and torch.equal(ms, runs[0][1])


def test_graph_replays():
    """Captured once, replayed over changing queries, lengths and tables."""
    m = R.to_gpu(R.make([800, 5, 0, 1200], 2, 128, 16, BF16, heads=8, seed=31), S)
    ws = S.KVWorkspace(m.cache, 8, mass=True)
    mass, out = torch.zeros(4, 2, 1200, device=DEV), torch.empty_like(m.gq)
    lens = [[800, 5, 0, 1200], [1, 0, 0, 900], [0, 0, 0, 0], [300, 5, 0, 17]]
    refs = []
    for k, ln in enumerate(lens):
        m.glens.copy_(torch.tensor(ln, dtype=torch.int32))
        rm = torch.zeros_like(mass)
        refs.append((m.cache.attend(m.gq * (k + 1), ws, mass=rm, window=500, sinks=3).clone(), rm))
    q = m.gq.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.cache.attend(q, ws, out=out, mass=mass, window=500, sinks=3)
    for rep in range(8):
        k = rep % len(lens)
        m.glens.copy_(torch.tensor(lens[k], dtype=torch.int32))
        q.copy_(m.gq * (k + 1))
        mass.zero_()
        out.fill_(3)
        ws.buf.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), refs[k][0].view(torch.int16)), rep
        assert torch.equal(mass, refs[k][1]), rep
