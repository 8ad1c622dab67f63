"""The cache operators where a serving program can go wrong with them: bad
indices, streams, captured graphs, caches past 32 bits of bytes, many and no
sequences, strided results, scores that rise along a prompt.  Tolerances are
those of tests/test_gpu_kv4.py."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_fp8_b200 as fp8mm
from tests import gpu_util as gu

from tests.test_gpu_kv4 import BF16_WEIGHTS, _check_attention, _filled, _i32, _kv

pytestmark = pytest.mark.gpu
INDEX, POSITION, SEQUENCE, PAGE = 2, 16, 17, 18               # of the device error word


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert fp8mm.last_device_error() == 0


def _error(site):
    word = fp8mm.last_device_error()
    assert (word & 0xFF, word >> 8 & 0xFF) == (INDEX, site)


def _workspace(dim):
    return torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")


def _queries(n, heads, dim, seed=1):
    return torch.randn(n, heads, dim, generator=torch.Generator().manual_seed(seed)).bfloat16()


# new tokens per sequence: a decode step, and chunks that the kernel for many rows takes
STEPS = [([1, 1, 1], 4, 2), ([70, 64, 70], 4, 2)]


@pytest.mark.parametrize("new,hq,hk", STEPS)
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_bad_page_ids(new, hq, hk, bad):
    """Recorded; the other sequences are as without it, and the cache as it was where pages have no place."""
    dim, lengths = 64, [100, 130, 80]
    cache, table, own = _filled(np.random.default_rng(4), lengths, 16, hk, dim, 3)
    table[1, 2] = bad
    if bad > 0:
        table[1, 2] = cache.data.shape[0]
    dev, cu = cache.data.cuda(), np.concatenate([[0], np.cumsum(new)]).tolist()
    q = _queries(cu[-1], hq, dim)
    for ws in (_workspace(dim), None):
        out = fp8mm.mxfp4_kv_attention(q.cuda(), dev, _i32(table), _i32(lengths), 16, cu_seqlens=_i32(cu), workspace=ws)
        _error(PAGE)
        lim = BF16_WEIGHTS if ws is not None and new[0] > 1 else 2.0 ** -10
        for s in (0, 2):
            rows = slice(cu[s], cu[s + 1])
            _check_attention(out[rows], None, q[rows], cache, [own[s]], [lengths[s]], [0, new[s]], dim ** -0.5, lim)
    k, v = (torch.zeros(130, hk, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k.fill_(7)
    fp8mm.mxfp4_kv_gather(dev, _i32(table[1:2]), _i32([0, 130]), 16, dim, 130, k=k, v=v)
    _error(PAGE)
    want = cache.read(own[1], 130)[0].bfloat16()
    assert torch.equal(k[:32].cpu(), want[:32]) and torch.equal(k[48:].cpu(), want[48:]) and (k[32:48] == 7).all()
    x = torch.ones(60, hk, dim, dtype=torch.bfloat16, device="cuda")
    fp8mm.mxfp4_kv_append(x[:16], x[:16], dev, _i32(table[1:2]), _i32([48]), 16, cu_seqlens=_i32([0, 16]))
    _error(PAGE)
    fp8mm.mxfp4_kv_append(x[:1], x[:1], dev, _i32(table[:1, :2]), _i32([33]), 16)     # behind the table
    _error(PAGE)
    assert torch.equal(dev.cpu(), cache.data)


@pytest.mark.parametrize("new,hq,hk", STEPS)
def test_bad_bounds_and_lengths(new, hq, hk):
    dim, lengths = 128, [100, 130, 80]
    cache, table, own = _filled(np.random.default_rng(4), lengths, 16, hk, dim, 3)
    dev, cu = cache.data.cuda(), np.concatenate([[0], np.cumsum(new)]).tolist()
    q, ws = _queries(cu[-1], hq, dim).cuda(), _workspace(dim)
    run = lambda lens, cu, out=None: fp8mm.mxfp4_kv_attention(q, dev, _i32(table), _i32(lens), 16, cu_seqlens=_i32(cu),
                                                              workspace=ws, out=out)
    good = run(lengths, cu)
    assert fp8mm.last_device_error() == 0
    out = torch.full_like(good, 5)
    run(lengths, [cu[0], cu[1], cu[2], cu[3] + 1], out)                                # past the rows
    _error(SEQUENCE)
    assert torch.equal(out[:cu[2]], good[:cu[2]]) and (out[cu[2]:] == 5).all()
    out = torch.full_like(good, 5)
    run(lengths, [cu[0], cu[2], cu[1], cu[3]], out)                                    # falling
    _error(SEQUENCE)
    run([100, 1 << 30, 80], cu)                                                        # longer than its pages
    _error(SEQUENCE)
    run([100, -5, 80], cu)
    _error(SEQUENCE)
    # rows that count many times
    n, rows = 3000, cu[-1]
    out = torch.full_like(good, 5)
    fp8mm.mxfp4_kv_attention(q, dev, _i32(table[:1]).expand(n, -1).contiguous(), _i32([100] * n), 16,
                             cu_seqlens=_i32([0, 0, rows] * (n // 3) + [0]), workspace=ws, out=out)
    _error(SEQUENCE)
    x = torch.ones(rows, hk, dim, dtype=torch.bfloat16, device="cuda")
    fp8mm.mxfp4_kv_append(x, x, dev, _i32(table), _i32([0, 0, 0]), 16, cu_seqlens=_i32(cu))            # padding: nothing
    assert fp8mm.last_device_error() == 0
    fp8mm.mxfp4_kv_append(x[:2], x[:2], dev, _i32(table[:1]), _i32([1]), 16, cu_seqlens=_i32([0, 2]))  # begins at -1
    _error(SEQUENCE)
    fp8mm.mxfp4_kv_append(x, x, dev, _i32(table[:1]), _i32([90]), 16, cu_seqlens=_i32([0, rows + 1]))  # past the rows
    _error(SEQUENCE)
    assert torch.equal(dev.cpu(), cache.data)
    k = torch.full((20, hk, dim), 7, dtype=torch.bfloat16, device="cuda")
    fp8mm.mxfp4_kv_gather(dev, _i32(table[:1]), _i32([0, 20]), 16, dim, 20, starts=_i32([-3]), k=k)
    _error(SEQUENCE)
    assert (k == 7).all()


def test_bad_positions():
    q, k = _queries(4, 2, 64).cuda(), _queries(4, 1, 64, 2).cuda()
    table = torch.cat([torch.ones(10, 32), torch.zeros(10, 32)], 1).cuda()
    qo, ko = torch.full_like(q, 5), torch.full_like(k, 5)
    fp8mm.qk_norm_rope(q, k, table, _i32([0, 10, -1, 9]), q_out=qo, k_out=ko)
    _error(POSITION)
    for x, y in ((q, qo), (k, ko)):
        assert torch.equal(y[[0, 3]], x[[0, 3]]) and (y[1:3] == 5).all()               # an angle of 0 turns nothing


@pytest.mark.parametrize("new,hq,hk", STEPS + [([1, 1, 1], 32, 1)])
def test_graph_replays_with_other_lengths(new, hq, hk):
    """One step captured, replayed over changed lengths and pages; two graphs share a workspace, one after the other."""
    dim, rng = 128, np.random.default_rng(9)
    cache, table, own = _filled(rng, [600, 90, 300], 16, hk, dim, 5)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q, lens, tab, dev, ws = _queries(cu[-1], hq, dim), _i32([1, 1, 1]), _i32(table), cache.data.cuda(), _workspace(dim)
    qd, cud = q.cuda(), _i32(cu)
    outs = [torch.empty_like(qd) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for out in outs:
        fp8mm.mxfp4_kv_attention(qd, dev, tab, lens, 16, cu_seqlens=cud, out=out, workspace=ws, stream=side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            fp8mm.mxfp4_kv_attention(qd, dev, tab, lens, 16, cu_seqlens=cud, out=out, workspace=ws)
        graphs.append(g)
    lim = BF16_WEIGHTS if new[0] > 1 else 2.0 ** -10
    for lengths in ([600, 90, 300], [0, 64, 17], [599, 70, 299]):
        lens.copy_(_i32(lengths))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(*outs)
        _check_attention(outs[0], None, q, cache, own, lengths, cu, dim ** -0.5, lim)


def test_a_whole_step_in_a_graph():
    """Norm, append, attention captured once; each replay is one token more."""
    dim, hq, hk, rng = 64, 4, 2, np.random.default_rng(2)
    cache, table, own = _filled(rng, [40, 17], 16, hk, dim, 8)
    g = torch.Generator().manual_seed(5)
    qkv = [torch.randn(2, hq + 2 * hk, dim, generator=g).bfloat16() for _ in range(4)]
    ang = torch.arange(100, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    x, lens, pos, tab, dev, ws = qkv[0].cuda(), _i32([40, 17]), _i32([39, 16]), _i32(table), cache.data.cuda(), _workspace(dim)
    out = torch.empty(2, hq, dim, dtype=torch.bfloat16, device="cuda")

    def step():
        q, k = fp8mm.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], cs, pos)
        fp8mm.mxfp4_kv_append(k, x[:, hq + hk:], dev, tab, lens, 16)
        fp8mm.mxfp4_kv_attention(q, dev, tab, lens, 16, out=out, workspace=ws)

    step()                                                     # rewrites the last token of each sequence
    torch.cuda.synchronize()
    dev.copy_(cache.data)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = cache.data.cuda()
    for i, y in enumerate(qkv):
        x.copy_(y)
        lens.copy_(_i32([40 + i, 17 + i]))
        pos.copy_(_i32([39 + i, 16 + i]))
        graph.replay()
        q, k = fp8mm.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], cs, pos)
        fp8mm.mxfp4_kv_append(k, x[:, hq + hk:], want, tab, lens, 16)
        torch.cuda.synchronize()
        assert torch.equal(dev, want)
        assert torch.equal(out, fp8mm.mxfp4_kv_attention(q, want, tab, lens, 16, workspace=ws))


@pytest.mark.parametrize("new,hq,hk", STEPS)
def test_another_stream(new, hq, hk):
    """Work on a given stream, behind what that stream already does."""
    dim, lengths = 64, [100, 130, 80]
    cache, table, own = _filled(np.random.default_rng(4), lengths, 16, hk, dim, 3)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q, dev, tab, ws = _queries(cu[-1], hq, dim), cache.data.cuda(), _i32(table), _workspace(dim)
    qd, late, lens, cud = q.cuda(), torch.zeros_like(dev), _i32(lengths), _i32(cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(8):
            busy = busy @ busy * 1e-3
        late.copy_(dev)
    out = fp8mm.mxfp4_kv_attention(qd, late, tab, lens, 16, cu_seqlens=cud, workspace=ws, stream=side)
    side.synchronize()
    _check_attention(out, None, q, cache, own, lengths, cu, dim ** -0.5, BF16_WEIGHTS if new[0] > 1 else 2.0 ** -10)


@pytest.mark.parametrize("dim", [64, 128])
def test_caches_past_32_bits(dim):
    """Pages whose offsets in bytes and in elements pass 2^32: append, read back, attend with either kernel, copy."""
    hk, n = 2, 150
    size = fp8mm.mxfp4_kv_page_bytes(64, hk, dim)
    stride = (1 << 31) + 4096
    room = torch.empty(3 * stride + size, dtype=torch.uint8, device="cuda")
    cache = room.as_strided((4, size), (stride, 1))
    near = torch.zeros(4, size, dtype=torch.uint8, device="cuda")
    cache.zero_()
    table = _i32([[3, 2, 1]])
    k, v = (x.cuda() for x in _kv(n, hk, dim, 4))
    for c in (cache, near):
        fp8mm.mxfp4_kv_append(k, v, c, table, _i32([n]), 64, cu_seqlens=_i32([0, n]))
    assert all(torch.equal(cache[i], near[i]) for i in range(4))
    q, ws = _queries(n, 4, dim).cuda(), _workspace(dim)
    for rows in (1, n):
        args = (table, _i32([n]), 64, _i32([0, rows]))
        a, b = (fp8mm.mxfp4_kv_attention(q[:rows], c, *args, workspace=ws) for c in (cache, near))
        assert torch.equal(a, b)
    a, b = (fp8mm.mxfp4_kv_gather(c, table, _i32([0, n]), 64, dim, n) for c in (cache, near))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    fp8mm.kv_copy_pages(cache, [3], [0])
    assert torch.equal(cache[0], near[3])


@pytest.mark.parametrize("dim,hq,hk", [(128, 4, 1), (64, 8, 2)])
def test_many_sequences(dim, hq, hk):
    """More sequences than a CTA has threads, most short, some empty, some long: each as on its own."""
    rng = np.random.default_rng(6)
    lengths = [int(x) for x in rng.integers(0, 40, 700)]
    lengths[5], lengths[350], lengths[699] = 900, 1500, 333
    cache, table, own = _filled(rng, lengths, 16, hk, dim, 12)
    q = _queries(700, hq, dim)
    out = fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32(lengths), 16, workspace=_workspace(dim))
    _check_attention(out, None, q, cache, own, lengths, range(701), dim ** -0.5)


def test_no_sequences_and_no_rows():
    cache = torch.zeros(3, fp8mm.mxfp4_kv_page_bytes(16, 2, 64), dtype=torch.uint8, device="cuda")
    none, q, x = _i32([]), _queries(5, 4, 64).cuda(), _queries(5, 2, 64).cuda()
    empty = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 5)
    fp8mm.mxfp4_kv_attention(q, cache, empty, none, 16, cu_seqlens=_i32([0]), out=out, workspace=_workspace(64))
    fp8mm.mxfp4_kv_append(x, x, cache, empty, none, 16, cu_seqlens=_i32([0]))
    fp8mm.mxfp4_kv_append(x[:0], x[:0], cache, empty, none, 16)
    k, v = fp8mm.mxfp4_kv_gather(cache, empty, _i32([0]), 16, 64, 0)
    assert (out == 5).all() and k.shape == v.shape == (0, 2, 64) and not cache.any()
    assert fp8mm.mxfp4_kv_attention(q[:0], cache, empty, none, 16).shape == (0, 4, 64)
    # sequences without tokens and pages: zeros
    out = fp8mm.mxfp4_kv_attention(q, cache, torch.zeros(5, 0, dtype=torch.int32, device="cuda"), _i32([0] * 5), 16)
    assert not out.any()
    fp8mm.kv_copy_pages(cache, [], [])


@pytest.mark.parametrize("new,hq,hk", STEPS)
def test_strided_results(new, hq, hk):
    """Results into slices of a wider buffer, whose other columns and rows stay; the same call twice gives the same bits."""
    dim, lengths = 64, [1000, 130, 80]
    cache, table, own = _filled(np.random.default_rng(4), lengths, 48, hk, dim, 3)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q, dev, ws = _queries(cu[-1], hq, dim), cache.data.cuda(), _workspace(dim)
    wide = torch.full((cu[-1] + 2, hq + 2, dim + 8), 5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((cu[-1], hq + 3), 5.0, device="cuda")
    first = None
    for _ in range(3):
        out = wide[:cu[-1], 1:hq + 1, 8:]
        fp8mm.mxfp4_kv_attention(q.cuda(), dev, _i32(table), _i32(lengths), 48, cu_seqlens=_i32(cu), out=out,
                                 lse=lse[:, :hq], workspace=ws)
        first = out.clone() if first is None else first
        assert torch.equal(first, out)
    _check_attention(first, lse[:, :hq], q, cache, own, lengths, cu, dim ** -0.5, BF16_WEIGHTS if new[0] > 1 else 2.0 ** -10)
    out.fill_(5)
    assert (wide == 5).all() and (lse[:, hq:] == 5).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 96])
@pytest.mark.parametrize("low,high", [(-50.0, 50.0), (50.0, -50.0), (0.0, 0.0)])
def test_scores_that_rise_along_a_prompt(dim, low, high, size):
    """Scores from `low` to `high` (natural units) along 700 tokens: rows whose first tokens' maximum is far below
    the last's, and far above; values of any size."""
    n, rows, heads = 700, 130, 2

    def make(length, h, d, seed):
        k, v = _kv(length, h, d, seed)
        ramp = torch.linspace(low, high, length)[:, None, None]
        k = 0.02 * k
        k[..., :32] = (ramp / 32).expand(length, h, 32).bfloat16()
        return k, v * size

    cache, table, own = _filled(np.random.default_rng(3), [n], 64, 1, dim, 9, make)
    q = _queries(rows, heads, dim)
    q[..., :32] = 1
    lse = torch.empty(rows, heads, device="cuda")
    out = fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32([n]), 64, cu_seqlens=_i32([0, rows]),
                                   scale=1.0, lse=lse, workspace=_workspace(dim))
    _check_attention(out, lse, q, cache, own, [n], [0, rows], 1.0, BF16_WEIGHTS)


def test_a_forked_and_compacted_pool():
    """A pool's forks, frees and compaction with the copies they ask for: every sequence reads what it wrote."""
    dim, hk, ps, layers = 64, 2, 16, 2
    pool = fp8mm.KvPagePool(20, ps)
    cache = torch.zeros(layers, 20, fp8mm.mxfp4_kv_page_bytes(ps, hk, dim), dtype=torch.uint8, device="cuda")
    k, v = (x.cuda() for x in _kv(80, hk, dim, 2))

    def write(pages, at, n):                                   # tokens at .. at + n of k, v behind at tokens
        for layer in cache:
            fp8mm.mxfp4_kv_append(k[at:at + n], v[at:at + n], layer, _i32([pages]), _i32([at + n]), ps, cu_seqlens=_i32([0, n]))

    def reads(pages, n):
        got = [fp8mm.mxfp4_kv_gather(layer, _i32([pages]), _i32([0, n]), ps, dim, n) for layer in cache]
        return [t for pair in got for t in pair]

    first = pool.allocate(2)
    a = pool.allocate(pool.pages_for(40))
    write(a, 0, 40)
    before = reads(a, 40)
    b, src, dst = pool.fork(a, 40)
    fp8mm.kv_copy_pages(cache, src, dst)
    b += pool.allocate(pool.pages_for(70) - len(b))
    write(b, 40, 30)                                           # the fork goes on; a keeps its own last page
    assert all(torch.equal(x, y) for x, y in zip(before, reads(a, 40)))
    longer = reads(b, 70)
    assert all(torch.equal(x, y[:40]) for x, y in zip(before, longer))
    pool.free(first)
    src, dst, moved = pool.compact()
    assert src
    fp8mm.kv_copy_pages(cache, src, dst)
    a, b = ([moved.get(p, p) for p in x] for x in (a, b))
    cache[:, pool.num_pages - pool.free_pages:] = 255          # what is free may hold anything
    assert all(torch.equal(x, y) for x, y in zip(before, reads(a, 40)))
    assert all(torch.equal(x, y) for x, y in zip(longer, reads(b, 70)))


@pytest.mark.parametrize("new,hq,hk", STEPS)
@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_scales_below_and_at_zero(new, hq, hk, scale):
    dim, lengths = 64, [100, 130, 80]
    cache, table, own = _filled(np.random.default_rng(4), lengths, 16, hk, dim, 3)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q, lse = _queries(cu[-1], hq, dim), torch.empty(cu[-1], hq, device="cuda")
    for ws in (_workspace(dim), None):
        out = fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32(lengths), 16, cu_seqlens=_i32(cu),
                                       scale=scale, lse=lse, workspace=ws)
        _check_attention(out, lse, q, cache, own, lengths, cu, scale,
                         BF16_WEIGHTS if ws is not None and new[0] > 1 else 2.0 ** -10)
