"""Batches of the cache operators: bounds that do not begin at row 0, lengths
that do not fit, many sequences, tables wider than 32 bits of work, single rows
of any stride, results over the queries, workspaces that were not zeroed, calls
at once on several streams.
Tolerances are those of tests/test_gpu_kv4.py."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_fp8_b200 as fp8mm
from tests import gpu_util as gu
from tests import kv4_ref as ref
from tests.test_gpu_kv4 import BF16_WEIGHTS, _check_attention, _filled, _i32, _kv, _tables

pytestmark = pytest.mark.gpu
INDEX, WORKSPACE = 2, 3                                        # kinds of the device error word
POSITION, SEQUENCE = 16, 17                                    # and places


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert fp8mm.last_device_error() == 0


def _workspace(dim):
    return torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")


def _queries(n, heads, dim, seed=1):
    return torch.randn(n, heads, dim, generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("first", [1, 5, 40])
@pytest.mark.parametrize("new", [[1, 3, 0, 1], [70, 64, 1, 90]])
def test_bounds_that_begin_behind_row_0(first, new):
    """Rows before cu_seqlens[0] belong to no sequence: not read, results as they were, no error."""
    dim, hk, hq, ps = 64, 2, 4, 16
    rng = np.random.default_rng(4)
    old = [20, 7, 33, 0]
    lengths = [a + b for a, b in zip(old, new)]
    cache, table, own = _filled(rng, lengths, ps, hk, dim, 3)
    cu = (first + np.concatenate([[0], np.cumsum(new)])).tolist()
    rows = cu[-1] + 2
    k, v = _kv(rows, hk, dim, 9)
    k[:first], v[:first] = float("nan"), float("nan")
    (kc, ke), (vc, ve) = ref.quantize(torch.nan_to_num(k)), ref.quantize(torch.nan_to_num(v))
    dev = cache.data.cuda()
    for s, n in enumerate(new):
        for t in range(n):
            r, pos = cu[s] + t, old[s] + t
            cache.write(own[s][pos // ps], pos % ps, kc[r], ke[r], vc[r], ve[r])
    fp8mm.mxfp4_kv_append(k.cuda(), v.cuda(), dev, _i32(table), _i32(lengths), ps, cu_seqlens=_i32(cu))
    assert fp8mm.last_device_error() == 0
    assert torch.equal(dev.cpu(), cache.data)
    gk, gv = (torch.full((rows, hk, dim), 7, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fp8mm.mxfp4_kv_gather(dev, _i32(table), _i32(cu), ps, dim, rows, starts=_i32(old), k=gk, v=gv)
    assert fp8mm.last_device_error() == 0
    for got, codes, e in ((gk, kc, ke), (gv, vc, ve)):
        want = ref.value(codes, e).bfloat16()
        assert torch.equal(got[first:cu[-1]].cpu(), want[first:cu[-1]]) and (got[:first] == 7).all() and (got[cu[-1]:] == 7).all()
    q = _queries(rows, hq, dim)
    for ws in (_workspace(dim), None):
        out = torch.full((rows, hq, dim), 5, dtype=torch.bfloat16, device="cuda")
        fp8mm.mxfp4_kv_attention(q.cuda(), dev, _i32(table), _i32(lengths), ps, cu_seqlens=_i32(cu), out=out, workspace=ws)
        many = ws is not None and -(-rows // 4) * 2 >= 96
        _check_attention(out, None, q, cache, own, lengths, cu, dim ** -0.5, BF16_WEIGHTS if many else 2.0 ** -10)
        assert (out[:first] == 5).all() and (out[cu[-1]:] == 5).all()


@pytest.mark.parametrize("new,hq,hk", [([1, 1, 1], 4, 2), ([70, 64, 70], 4, 2)])
@pytest.mark.parametrize("bad", [113, 1 << 30, (1 << 31) - 1, -1, -(1 << 31)])
def test_lengths_that_do_not_fit(new, hq, hk, bad):
    """A sequence whose length is negative, or longer than its row of the page table, is recorded and skipped."""
    dim, lengths = 64, [100, 112, 80]
    cache, table, own = _filled(np.random.default_rng(4), lengths, 16, hk, dim, 3)
    dev, cu = cache.data.cuda(), np.concatenate([[0], np.cumsum(new)]).tolist()
    q = _queries(cu[-1], hq, dim)
    for ws in (_workspace(dim), None):
        out = torch.full((cu[-1], hq, dim), 5, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((cu[-1], hq), 5.0, device="cuda")
        fp8mm.mxfp4_kv_attention(q.cuda(), dev, _i32(table), _i32([100, bad, 80]), 16, cu_seqlens=_i32(cu), out=out, lse=lse,
                                 workspace=ws)
        word = fp8mm.last_device_error()
        assert (word & 0xFF, word >> 8 & 0xFF) == (INDEX, SEQUENCE)
        assert (out[cu[1]:cu[2]] == 5).all() and (lse[cu[1]:cu[2]] == 5).all()
        lim = BF16_WEIGHTS if ws is not None and new[0] > 1 else 2.0 ** -10
        for s in (0, 2):
            rows = slice(cu[s], cu[s + 1])
            _check_attention(out[rows], lse[rows], q[rows], cache, [own[s]], [lengths[s]], [0, new[s]], dim ** -0.5, lim)


@pytest.mark.parametrize("batch,most", [(40, 5), (700, 4), (1500, 3)])
def test_append_and_gather_of_many_sequences(batch, most):
    """More sequences than a warp, and than its square, searches at once, with empty ones at either end and in runs."""
    rng = np.random.default_rng(batch)
    new = rng.integers(0, most, batch)
    new[[0, 1, batch - 1]] = 0
    new[batch // 3:batch // 3 + 37] = 0
    new[batch // 2] = 61
    old = np.where(new > 0, rng.integers(0, 20, batch), 0)
    lengths = (old + new).tolist()
    table, own, pages = _tables(rng, lengths, 16)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    cache = ref.Cache(pages, 16, 1, 64, seed=5)
    dev = cache.data.cuda()
    k, v = _kv(cu[-1] + 3, 1, 64, 2)
    (kc, ke), (vc, ve) = ref.quantize(k), ref.quantize(v)
    for s in range(batch):
        for t in range(new[s]):
            r, pos = cu[s] + t, int(old[s]) + t
            cache.write(own[s][pos // 16], pos % 16, kc[r], ke[r], vc[r], ve[r])
    fp8mm.mxfp4_kv_append(k.cuda(), v.cuda(), dev, _i32(table), _i32(lengths), 16, cu_seqlens=_i32(cu))
    assert torch.equal(dev.cpu(), cache.data)
    got = fp8mm.mxfp4_kv_gather(dev, _i32(table), _i32(cu), 16, 64, cu[-1], starts=_i32(old.tolist()))
    for x, codes, e in zip(got, (kc, vc), (ke, ve)):
        assert torch.equal(x.cpu(), ref.value(codes, e).bfloat16()[:cu[-1]])


@pytest.mark.parametrize("batch,new,hq", [(600, 2, 2), (600, 3, 8), (300, 6, 16)])
def test_attention_of_many_ragged_sequences(batch, new, hq):
    """Several sequences to a strip of the plan: ragged ones, some without rows; the last shape on the kernel for many rows."""
    rng = np.random.default_rng(batch + new)
    count = rng.integers(0, 2 * new + 1, batch)
    count[:3] = 0
    count[-1] = 5 * batch * new // 100 + 1
    total = int(count.sum())
    lengths = (count + rng.integers(0, 50, batch)).tolist()
    lengths[7] = 700
    cache, table, own = _filled(rng, lengths, 32, 1, 64, 12)
    cu = np.concatenate([[0], np.cumsum(count)]).tolist()
    q = _queries(total, hq, 64)
    for ws in (_workspace(64), None):
        out = fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32(lengths), 32, cu_seqlens=_i32(cu), workspace=ws)
        many = ws is not None and -(-total // batch) * hq >= 96
        assert many == (ws is not None and hq == 16)
        _check_attention(out, None, q, cache, own, lengths, cu, 0.125, BF16_WEIGHTS if many else 2.0 ** -10)


@pytest.mark.parametrize("hq", [16, 128])
def test_tables_wide_enough_for_coarse_units(hq):
    """A page table with room for 2^31 tokens a sequence: the plan's units stand for several steps each."""
    dim, hk, ps, batch = 64, 16, 4096, 2
    most = (2 ** 31 - 1) // ps
    lengths, rows = [5000, 9000], [1, 1]
    k, v = _kv(sum(lengths), hk, dim, 3)
    cache = torch.zeros(6, fp8mm.mxfp4_kv_page_bytes(ps, hk, dim), dtype=torch.uint8, device="cuda")
    pages = [[4, 1], [0, 5, 2]]
    wide = torch.full((batch, most), -1, dtype=torch.int32, device="cuda")
    for s, p in enumerate(pages):
        wide[s, :len(p)] = _i32(p)
    narrow = wide[:, :3].contiguous()
    cu = _i32([0, 5000, 14000])
    fp8mm.mxfp4_kv_append(k.cuda(), v.cuda(), cache, wide, _i32(lengths), ps, cu_seqlens=cu)
    got = fp8mm.mxfp4_kv_gather(cache, narrow, cu, ps, dim, 14000)
    want = [ref.value(*ref.quantize(x)) for x in (k, v)]
    assert all(torch.equal(a.cpu(), b.bfloat16()) for a, b in zip(got, want))
    q = _queries(2, hq, dim)
    steps, tiles = (2 ** 31 - 1) // 32 + 7, (2 * hq // hk / 4 + 2) * hk
    assert steps * tiles > 2e9                                  # units of one step would pass 31 bits
    for table in (wide, narrow):
        out = fp8mm.mxfp4_kv_attention(q.cuda(), cache, table, _i32(lengths), ps, workspace=_workspace(dim)).double().cpu()
        for s, (a, b) in enumerate(((0, 5000), (5000, 14000))):
            w, mag, _ = ref.attention(q[s:s + 1], want[0][a:b], want[1][a:b], dim ** -0.5)
            assert ((out[s:s + 1] - w).abs() <= 2.0 ** -8 * w.abs() + (2.0 ** -10 + 2.0 ** -16) * mag).all()


def test_single_rows_and_heads_of_any_stride():
    """The stride of a dimension of one element says nothing: it is not checked."""
    dim, ps = 64, 16
    odd = lambda x, stride: x.contiguous().as_strided(x.shape, stride)
    g = torch.Generator().manual_seed(3)
    cs = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).cuda()
    q, k, v = (torch.randn(1, h, dim, generator=g).bfloat16().cuda() for h in (2, 1, 1))
    cache = torch.zeros(1, fp8mm.mxfp4_kv_page_bytes(ps, 1, dim), dtype=torch.uint8, device="cuda")
    table, lens = _i32([[0]]), _i32([1])
    q1, k1, v1 = odd(q, (3, dim, 1)), odd(k, (0, 5, 1)), odd(v, (1, 0, 1))
    qo, ko = fp8mm.qk_norm_rope(q1, k1, odd(cs, (0, 1)), _i32([0]), q_out=torch.empty_like(q).as_strided(q.shape, (0, dim, 1)))
    assert torch.equal(qo, q) and torch.equal(ko, k)
    one = odd(cache, (1, 1))
    fp8mm.mxfp4_kv_append(k1, v1, one, odd(table, (0, 1)), lens, ps)
    k2, v2 = (torch.empty_like(k).as_strided(k.shape, (3, 3, 1)) for _ in range(2))
    fp8mm.mxfp4_kv_gather(one, table, _i32([0, 1]), ps, dim, 1, k=k2, v=v2)
    assert torch.equal(v2.cpu(), ref.value(*ref.quantize(v.cpu())).bfloat16())
    out = torch.empty_like(q).as_strided(q.shape, (0, dim, 1))
    fp8mm.mxfp4_kv_attention(q1, one, table, lens, ps, out=out)
    assert torch.equal(out, v2.expand(1, 2, dim))
    layers = torch.arange(64, dtype=torch.uint8, device="cuda").view(1, 4, 16)
    fp8mm.kv_copy_pages(layers.as_strided(layers.shape, (5, 16, 1)), [0], [3])
    assert torch.equal(layers[0, 3], layers[0, 0])


@pytest.mark.parametrize("new,hq,hk", [([1, 1, 1], 4, 2), ([1, 1, 1], 32, 2), ([70, 64, 70], 4, 2)])
def test_results_over_the_queries(new, hq, hk):
    dim, lengths = 64, [1500, 130, 800]
    cache, table, own = _filled(np.random.default_rng(4), lengths, 16, hk, dim, 3)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q, dev, ws = _queries(cu[-1], hq, dim).cuda(), cache.data.cuda(), _workspace(dim)
    args = (dev, _i32(table), _i32(lengths), 16, _i32(cu))
    want = fp8mm.mxfp4_kv_attention(q, *args, workspace=ws)
    got = fp8mm.mxfp4_kv_attention(q, *args, workspace=ws, out=q)
    assert got is q and torch.equal(got, want)


def test_error_words_of_both_kinds_are_kept():
    """An expired wait of a GEMM and a bad position stand side by side: each is reported, one after the other."""
    assert fp8mm.last_device_error() == 0
    a = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    cs = torch.zeros(1, 64, device="cuda")
    for _ in range(2):
        fp8mm.qk_norm_rope(a, a, cs, _i32([7]))
        L = fp8mm.fp8mm.lib()
        assert L.fp8mm_selftest_wait_timeout(2000, None) == fp8mm.fp8mm.FP8MM_ERR_DEVICE
        word = fp8mm.last_device_error()
        assert (word & 0xFF, word >> 8 & 0xFF) == (INDEX, POSITION)
        assert fp8mm.last_device_error() == 0


def test_lengths_next_to_2_to_the_31():
    """A table with room for 2^31 - 16 tokens (of one page, repeated): lengths within 64 of 2^31, whose positions would
    pass an int, are recorded and nothing is done."""
    dim, ps, hk = 64, 16, 1
    most = (2 ** 31 - 1) // ps
    cache = torch.zeros(1, fp8mm.mxfp4_kv_page_bytes(ps, hk, dim), dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, most, dtype=torch.int32, device="cuda")
    assert most * ps > 2 ** 31 - 20
    bad = _i32([2 ** 31 - 20])
    q, x = _queries(200, 4, dim).cuda(), _queries(200, 1, dim).cuda()
    for rows, ws in ((1, None), (1, _workspace(dim)), (200, _workspace(dim))):
        out = torch.full_like(q, 5)
        fp8mm.mxfp4_kv_attention(q, cache, table, bad, ps, cu_seqlens=_i32([0, rows]), out=out, workspace=ws)
        word = fp8mm.last_device_error()
        assert (word & 0xFF, word >> 8 & 0xFF) == (INDEX, SEQUENCE) and (out == 5).all()
    fp8mm.mxfp4_kv_append(x, x, cache, table, bad, ps, cu_seqlens=_i32([0, 200]))
    word = fp8mm.last_device_error()
    assert (word & 0xFF, word >> 8 & 0xFF) == (INDEX, SEQUENCE) and not cache.any()


@pytest.mark.parametrize("new,hq,hk", [([1, 1, 1], 4, 2), ([70, 64, 70], 4, 2)])
@pytest.mark.parametrize("fill", [255, 1, "random"])
def test_workspaces_that_were_not_zeroed(new, hq, hk, fill):
    """Recorded, whatever the bytes say; with the counters zeroed the same workspace serves."""
    dim, lengths = 64, [3000, 130, 80]
    cache, table, own = _filled(np.random.default_rng(4), lengths, 16, hk, dim, 3)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q, ws = _queries(cu[-1], hq, dim), _workspace(dim)
    if fill == "random":
        ws.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(3))
    else:
        ws.fill_(fill)
    args = (q.cuda(), cache.data.cuda(), _i32(table), _i32(lengths), 16, _i32(cu))
    for _ in range(2):
        fp8mm.mxfp4_kv_attention(*args, workspace=ws)
        assert fp8mm.last_device_error() & 0xFF == WORKSPACE
    ws[:256] = 0
    for _ in range(2):
        out = fp8mm.mxfp4_kv_attention(*args, workspace=ws)
        _check_attention(out, None, q, cache, own, lengths, cu, dim ** -0.5, BF16_WEIGHTS if new[0] > 1 else 2.0 ** -10)


def test_calls_at_once_on_several_streams():
    """Attention of few and of many rows, each with its own workspace, norms, a product and an append into another cache,
    at once on four streams: the same bits as one after the other."""
    g = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    jobs = []
    for dim, hq, hk, new, length in ((64, 8, 2, 70, 2000), (128, 8, 2, 1, 3000)):
        batch, ps = 3, 64
        per = -(-length // ps)
        cache = torch.zeros(batch * per, fp8mm.mxfp4_kv_page_bytes(ps, hk, dim), dtype=torch.uint8, device="cuda")
        table = _i32(torch.randperm(batch * per, generator=torch.Generator().manual_seed(1)).view(batch, per).tolist())
        lens, rows = _i32([length, length - 700, 65]), [0, length, 2 * length - 700, 2 * length - 635]
        k, v, q = randn(rows[-1], hk, dim), randn(rows[-1], hk, dim), randn(new * batch, hq, dim)
        cu, ws, other = _i32([i * min(new, 65) for i in range(batch + 1)]), _workspace(dim), torch.zeros_like(cache)
        fp8mm.mxfp4_kv_append(k, v, cache, table, lens, ps, _i32(rows))
        out, cu_rows = torch.zeros_like(q), _i32(rows)
        jobs.append(lambda s, a=(q, cache, table, lens, ps, cu), o=out, w=ws: fp8mm.mxfp4_kv_attention(*a, out=o, workspace=w, stream=s))
        jobs.append(lambda s, a=(k, v, other, table, lens, ps, cu_rows): fp8mm.mxfp4_kv_append(*a, stream=s))
    x, cs, pos = randn(4096, 10, 128), torch.randn(4096, 128, device="cuda"), torch.arange(4096, dtype=torch.int32, device="cuda")
    qo, ko = torch.zeros_like(x[:, :8]), torch.zeros_like(x[:, 8:])
    jobs.append(lambda s: fp8mm.qk_norm_rope(x[:, :8], x[:, 8:], cs, pos, q_out=qo, k_out=ko, stream=s)[0])
    a, b = fp8mm.mxfp8_quantize(randn(512, 1024)), fp8mm.mxfp8_quantize(randn(1024, 1024))
    c = torch.zeros(512, 1024, dtype=torch.bfloat16, device="cuda")
    jobs.append(lambda s: fp8mm.mxfp8_gemm(*a, *b, c=c, stream=s))
    results, want = [], []
    for job in jobs:
        results.append(job(torch.cuda.current_stream()))
        torch.cuda.synchronize()
        want.append(results[-1].clone())
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(8):
        for r in results:
            r.zero_()
        torch.cuda.synchronize()
        for i, job in enumerate(jobs * 3):                     # a job stays on its stream
            job(streams[i % len(jobs) % 4])
        torch.cuda.synchronize()
        assert all(torch.equal(r, w) for r, w in zip(results, want))
