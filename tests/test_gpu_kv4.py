"""The MXFP4 paged key/value cache on the GPU (append, read back, attention,
page moves) and the norm and rotation before it, against 64-bit references on
the CPU (tests/kv4_ref.py).

Tolerances.  Bytes written and values read back are exact.  Attention: the
output's rounding to bf16 is at most 2^-8 of it; every weight is rounded to
f16 once (2^-11 of it), and a weight's other errors (fp32 scores of magnitude
up to a hundred, exp2 to 2^-22, fp32 sums) together stay below 2^-11 of it, so
the sum of weight * |v| counts with 2^-10.  A weight below 2^-26 of its block's
reference is an f16 subnormal: the product weight * 2^(e - E) * 2^12 is off by at
most 2^-25, that is 2^-37 in units of 2^E * |code|.  E is at most the largest
e + log2(weight) + 1 or the largest e, and weights are at most 2^2 of the running
maximum, so 2^E <= 2^3 * 2^e of some token, whose block has a value above 3 * 2^e: as
|code| <= 6, 2^E * |code| <= 2^4 * (largest |v| of the block).  The sum of weights is at
least 2^-2 in the same units (a maximum is set 2 above the score that moved it), so
n tokens are off by n * 2^-31 of it.  Norm and rotation: 2^-8 of the result,
and some fp32 roundings (2^-20) of the two terms of a rotated element."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_fp8_b200 as fp8mm
from tests import gpu_util as gu
from tests import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert fp8mm.last_device_error() == 0


def _kv(n, heads, dim, seed):
    g = torch.Generator().manual_seed(seed)
    chan = torch.exp(torch.randn(heads, dim, generator=g))
    return ((torch.randn(n, heads, dim, generator=g) * chan).bfloat16(),
            (torch.randn(n, heads, dim, generator=g) * 0.5).bfloat16())


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(rng, lengths, page_size, spare=2):
    """Scattered pages for each sequence: (table with -1 behind a sequence, pages of each, page count)."""
    counts = [-(-n // page_size) for n in lengths]
    ids = rng.permutation(sum(counts) + spare).tolist()
    own, table = [], np.full((len(lengths), max(counts + [1])), -1, dtype=np.int32)
    for s, c in enumerate(counts):
        own.append(ids[:c])
        table[s, :c] = ids[:c]
        ids = ids[c:]
    return table, own, sum(counts) + spare


def _filled(rng, lengths, page_size, heads, dim, seed, make=_kv):
    """A CPU cache holding `lengths` tokens of each sequence, its table, and the stored fp64 keys and values."""
    table, own, n = _tables(rng, lengths, page_size)
    cache = ref.Cache(n, page_size, heads, dim, seed)
    for s, length in enumerate(lengths):
        k, v = make(length, heads, dim, seed + 7 * s)
        (kc, ke), (vc, ve) = ref.quantize(k), ref.quantize(v)
        for t in range(length):
            cache.write(own[s][t // page_size], t % page_size, kc[t], ke[t], vc[t], ve[t])
    return cache, table, own


# rows of a head per sequence, on average, from which the tcgen05 kernel runs (with a workspace); it rounds weights to
# bf16 (2^-8 of each) where the other rounds them to f16
MANY_ROWS, BF16_WEIGHTS = 96, 2.0 ** -8 + 2.0 ** -11


def _check_attention(out, lse, q, cache, own, lengths, cu, scale, weights=2.0 ** -10):
    out, lse = out.double().cpu(), None if lse is None else lse.double().cpu()
    for s, length in enumerate(lengths):
        rows = slice(cu[s], cu[s + 1])
        k, v = cache.read(own[s], length) if length else (torch.zeros(0, cache.heads, cache.dim).double(),) * 2
        want, mag, wlse = ref.attention(q[rows], k, v, scale)
        top = v.abs().amax(0).unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1) if length else torch.zeros(cache.heads, cache.dim)
        top = top.repeat_interleave(q.shape[1] // cache.heads, 0)
        lim = 2.0 ** -8 * want.abs() + weights * mag + length * 2.0 ** -31 * top + 1e-37
        bad = (out[rows] - want).abs() / lim
        assert torch.isfinite(out[rows]).all() and (bad.numel() == 0 or bad.max() <= 1), (s, bad.max(), bad.argmax(), want.flatten()[bad.argmax()], out[rows].flatten()[bad.argmax()], lim.flatten()[bad.argmax()])
        if lse is not None:
            fine = torch.isfinite(wlse)
            assert torch.equal(fine, torch.isfinite(lse[rows])) and (lse[rows][~fine] < 0).all()
            assert ((lse[rows] - wlse)[fine].abs() <= 2.0 ** -14 * (1 + wlse[fine].abs())).all()


# ------------------------------------------------------------------ append and gather

def _append_all(cache, table, rng, steps, page_size, heads, dim, seed, strided=False):
    """Appends steps = [[new tokens of each sequence] per call] to `cache` (CPU) and its copy on the GPU."""
    dev = cache.data.cuda()
    own = [[int(p) for p in row if p >= 0] for row in table]
    at = [0] * len(own)
    for i, new in enumerate(steps):
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        k, v = _kv(cu[-1] + 3, heads, dim, seed + i)      # three rows of padding behind the last sequence
        (kc, ke), (vc, ve) = ref.quantize(k), ref.quantize(v)
        for s, n in enumerate(new):
            for t in range(n):
                r, pos = cu[s] + t, at[s] + t
                cache.write(own[s][pos // page_size], pos % page_size, kc[r], ke[r], vc[r], ve[r])
            at[s] += n
        if strided:                                       # slices of one projection's output
            qkv = torch.cat([torch.zeros(k.shape[0], 5 * dim).bfloat16(), k.flatten(1), v.flatten(1)], 1).cuda()
            kd = qkv[:, 5 * dim:(5 + heads) * dim].unflatten(1, (heads, dim))
            vd = qkv[:, (5 + heads) * dim:].unflatten(1, (heads, dim))
        else:
            kd, vd = k.cuda(), v.cuda()
        fp8mm.mxfp4_kv_append(kd, vd, dev, _i32(table), _i32(at), page_size, cu_seqlens=_i32(cu))
    return dev, own, at


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page_size", [16, 48, 64])
@pytest.mark.parametrize("steps", [[[1, 1, 1]] * 3, [[5, 0, 16], [12, 33, 1], [1, 1, 1]], [[100, 17, 31]]])
def test_append_writes_the_bytes_and_no_others(dim, page_size, steps):
    rng = np.random.default_rng(1)
    lengths = np.sum(steps, 0).tolist()
    table, _, n = _tables(rng, lengths, page_size)
    cache = ref.Cache(n, page_size, 3, dim, seed=5)
    dev, own, at = _append_all(cache, table, rng, steps, page_size, 3, dim, 11, strided=dim == 128)
    assert at == lengths
    assert torch.equal(dev.cpu(), cache.data)


def test_append_extreme_values():
    """Zeros, negative zeros, subnormals, the largest magnitudes, and every tie between two codes."""
    dim, heads = 128, 1
    x = torch.zeros(20, heads, dim)
    x[1] = -0.0
    x[2] = 1e-40
    x[3, :, ::2] = 3.3e38
    x[4] = 2.0 ** -126
    x[5, :, 5] = 1e-38
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for i, s in enumerate((1.0, 2.0 ** -20, 2.0 ** 60, 2.0 ** -120)):
        x[6 + i] = (ties.repeat(dim // 8) * s).view(1, dim)
        x[10 + i] = -x[6 + i]
    for i, m in enumerate((1.5, 1.5078125, 1.4921875, 1.0, 1.9921875)):      # block maxima at the exponent rule's edge
        x[14 + i, :, 0] = m
        x[14 + i, :, 1:] = m / 7
    x = x.bfloat16()
    cache = ref.Cache(2, 16, heads, dim)
    (c, e) = ref.quantize(x)
    for t in range(20):
        cache.write(t // 16, t % 16, c[t], e[t], c[t], e[t])
    dev = ref.Cache(2, 16, heads, dim).data.cuda()
    fp8mm.mxfp4_kv_append(x.cuda(), x.cuda(), dev, _i32([[0, 1]]), _i32([20]), 16, cu_seqlens=_i32([0, 20]))
    assert torch.equal(dev.cpu(), cache.data)
    k, v = fp8mm.mxfp4_kv_gather(dev, _i32([[0, 1]]), _i32([0, 20]), 16, dim, 20)
    want = ref.value(c, e).bfloat16()
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)


def test_append_padding_sequences_and_rows():
    """A padded decode batch: sequences of length 0 write nothing, with one row each."""
    cache = ref.Cache(3, 16, 2, 64, seed=2)
    before = cache.data.clone()
    k, v = _kv(3, 2, 64, 3)
    dev = cache.data.cuda()
    fp8mm.mxfp4_kv_append(k.cuda(), v.cuda(), dev, _i32([[-1], [2], [-1]]), _i32([0, 16, 0]), 16)
    (kc, ke), (vc, ve) = ref.quantize(k), ref.quantize(v)
    cache.write(2, 15, kc[1], ke[1], vc[1], ve[1])
    assert torch.equal(dev.cpu(), cache.data) and not torch.equal(before, cache.data)


@pytest.mark.parametrize("dim,page_size", [(64, 16), (128, 64), (128, 32)])
def test_gather(dim, page_size):
    rng = np.random.default_rng(4)
    lengths = [1, 130, 16, 0, 47]
    cache, table, own = _filled(rng, lengths, page_size, 2, dim, 9)
    dev = cache.data.cuda()
    for starts, counts in ((None, lengths), ([0, 3, 15, 0, 32], [1, 127, 1, 0, 15]), ([0, 129, 2, 0, 5], [0, 1, 14, 0, 42])):
        cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
        total = cu[-1] + 4                                # rows behind the last sequence stay as they were
        k = torch.full((total, 2, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        v = torch.full((total, 2, 2 * dim), 9.0, dtype=torch.bfloat16, device="cuda")
        fp8mm.mxfp4_kv_gather(dev, _i32(table), _i32(cu), page_size, dim, total, starts=None if starts is None else _i32(starts),
                              k=k, v=v[..., dim:])
        for s, n in enumerate(counts):
            a = 0 if starts is None else starts[s]
            if n:
                wk, wv = cache.read(own[s], a + n)
                assert torch.equal(k[cu[s]:cu[s + 1]].cpu(), wk[a:].bfloat16())
                assert torch.equal(v[cu[s]:cu[s + 1], :, dim:].cpu(), wv[a:].bfloat16())
        assert (k[cu[-1]:] == 7).all() and (v[..., :dim] == 9).all() and (v[cu[-1]:] == 9).all()


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page_size", [16, 64])
@pytest.mark.parametrize("q_heads,kv_heads", [(4, 1), (2, 2), (14, 2), (16, 1), (20, 1)])
def test_decode_attention(dim, page_size, q_heads, kv_heads):
    rng = np.random.default_rng(3)
    lengths = [1, 300, 0, 16, 17, 129]
    cache, table, own = _filled(rng, lengths, page_size, kv_heads, dim, 21)
    q = torch.randn(len(lengths), q_heads, dim, generator=torch.Generator().manual_seed(1)).bfloat16()
    ws = torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    for workspace in (ws, None, ws):
        lse = torch.empty(len(lengths), q_heads, device="cuda")
        out = fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32(lengths), page_size, lse=lse,
                                       workspace=workspace)
        _check_attention(out, lse, q, cache, own, lengths, range(len(lengths) + 1), dim ** -0.5)
    assert not ws.view(torch.int32)[:64].any()            # the counters are left at zero


@pytest.mark.parametrize("dim,q_heads,kv_heads", [(128, 8, 2), (64, 3, 1), (128, 6, 1), (128, 2, 2)])
@pytest.mark.parametrize("new,lengths", [([3, 1, 0, 8, 4], [200, 1, 50, 8, 2]), ([70, 5], [90, 150]), ([40, 33], [40, 32])])
def test_several_queries_are_causal(dim, q_heads, kv_heads, new, lengths):
    """Queries at the last positions, some sequences shorter than their queries (their first rows see nothing)."""
    rng = np.random.default_rng(8)
    cache, table, own = _filled(rng, lengths, 32, kv_heads, dim, 31)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    rows = cu[-1] + 2
    qkv = torch.randn(rows, (q_heads + 3) * dim, generator=torch.Generator().manual_seed(2)).bfloat16()
    q = qkv[:, 2 * dim:(q_heads + 2) * dim].unflatten(1, (q_heads, dim))
    ws = torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    qd = qkv.cuda()[:, 2 * dim:(q_heads + 2) * dim].unflatten(1, (q_heads, dim))
    for workspace in (ws, None):
        out = torch.full((rows, q_heads, dim), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows, q_heads), 5.0, device="cuda")
        fp8mm.mxfp4_kv_attention(qd, cache.data.cuda(), _i32(table), _i32(lengths), 32, cu_seqlens=_i32(cu), scale=0.2,
                                 out=out, lse=lse, workspace=workspace)
        many = workspace is not None and -(-rows // len(new)) * (q_heads // kv_heads) >= MANY_ROWS
        _check_attention(out, lse, q, cache, own, lengths, cu, 0.2, BF16_WEIGHTS if many else 2.0 ** -10)
        assert (out[cu[-1]:] == 5).all() and (lse[cu[-1]:] == 5).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(8, 2), (3, 3), (5, 1), (16, 1)])
@pytest.mark.parametrize("new,lengths", [([300], [300]), ([257, 1, 0, 130], [600, 400, 50, 100]), ([129, 128], [127, 1100])])
def test_chunks_of_prompts(dim, q_heads, kv_heads, new, lengths):
    """Many queries a sequence: no prefix, long prefixes, a sequence shorter than its queries, empty and single ones."""
    rng = np.random.default_rng(9)
    cache, table, own = _filled(rng, lengths, 64, kv_heads, dim, 61)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = torch.randn(cu[-1] + 1, q_heads, dim, generator=torch.Generator().manual_seed(4)).bfloat16()
    ws = torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    for scale in (dim ** -0.5, -0.3):
        out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], 5.0, device="cuda")
        for _ in range(2):                                 # twice on one workspace: the same bits
            before = out.clone()
            fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32(lengths), 64, cu_seqlens=_i32(cu),
                                     scale=scale, out=out, lse=lse, workspace=ws)
        assert torch.equal(before, out)
        _check_attention(out, lse, q, cache, own, lengths, cu, scale, BF16_WEIGHTS)
        assert (out[cu[-1]:] == 5).all() and (lse[cu[-1]:] == 5).all()
    assert not ws.view(torch.int32)[:64].any()


def _uneven(n, heads, dim, seed):
    """Value magnitudes over 40 binades between tokens and blocks, keys over 20, zero rows among them."""
    g = torch.Generator().manual_seed(seed)
    k, v = _kv(n, heads, dim, seed)
    k = k * torch.exp2(torch.randint(-18, 3, (n, 1, dim // 32), generator=g).float()).repeat_interleave(32, 2)
    v = v * torch.exp2(torch.randint(-20, 21, (n, heads, dim // 32), generator=g).float()).repeat_interleave(32, 2)
    v[::5] = 0
    k[3::7] = 0
    return k.bfloat16(), v.bfloat16()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sharp", [0.05, 4.0])
def test_uneven_magnitudes(dim, sharp):
    """Weights and value exponents far apart: per-block references follow what matters."""
    rng = np.random.default_rng(13)
    lengths = [513, 40]
    cache, table, own = _filled(rng, lengths, 64, 1, dim, 41, make=_uneven)
    q = (torch.randn(2, 4, dim, generator=torch.Generator().manual_seed(3)) * torch.tensor([1.0, 2.0 ** 40, 2.0 ** -60, 1.0]).view(1, 4, 1)).bfloat16()
    q[:, 3] = 0
    q[:, 1] = (q[:, 1].double() * 2.0 ** -40).bfloat16()
    out = fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32(lengths), 64, scale=sharp)
    _check_attention(out, None, q, cache, own, lengths, range(3), sharp)
    q = q.repeat_interleave(40, 0)                         # 40 queries a sequence, on the kernel for many
    ws = torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    out = fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32(lengths), 64, cu_seqlens=_i32([0, 40, 80]),
                                   scale=sharp, workspace=ws)
    _check_attention(out, None, q, cache, own, lengths, [0, 40, 80], sharp, BF16_WEIGHTS)


def test_outlier_value_with_no_weight():
    """One token whose values are 2^60 times the others' and whose weight is zero in fp32: the others' sum is kept."""
    dim, n = 128, 200
    k = torch.full((n, 1, dim), 0.5)
    v = torch.randn(n, 1, dim, generator=torch.Generator().manual_seed(5))
    k[::50], v[::50] = -24.0, v[::50] * 2.0 ** 60
    k, v = k.bfloat16(), v.bfloat16()
    rng = np.random.default_rng(14)
    cache, table, own = _filled(rng, [n], 16, 1, dim, 51, make=lambda *a: (k, v))
    q = torch.ones(1, 2, dim).bfloat16()
    out = fp8mm.mxfp4_kv_attention(q.cuda(), cache.data.cuda(), _i32(table), _i32([n]), 16, scale=1.0)
    _check_attention(out, None, q, cache, own, [n], range(2), 1.0)


# ------------------------------------------------------------------ pages

@pytest.mark.parametrize("layers,pages,nbytes", [(None, 5, 16), (3, 40, 1088 * 3), (2, 1300, 2176)])
def test_copy_pages(layers, pages, nbytes):
    g = torch.Generator().manual_seed(6)
    shape = (pages, nbytes + 32) if layers is None else (layers, pages, nbytes + 32)
    data = torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8)
    ids = torch.randperm(pages, generator=g)
    n = pages // 2
    src, dst = ids[:n].clone(), ids[n:2 * n]
    src[-1] = src[0]                                       # a page may be copied twice
    dev = data.cuda()
    fp8mm.kv_copy_pages(dev[..., :nbytes], src, dst.tolist())
    want = data.clone()
    want[..., dst, :nbytes] = data[..., src, :nbytes]
    assert torch.equal(dev.cpu(), want)


# ------------------------------------------------------------------ norm and rotation

@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (128, 128), (128, 16), (256, 256), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 1), (37, 14, 2), (700, 5, 1)])
def test_norm_rope(dim, rot, interleaved, tokens, hq, hk):
    g = torch.Generator().manual_seed(tokens + dim)
    qkv = (torch.randn(tokens, (hq + 2 * hk) * dim, generator=g) * 3).bfloat16()
    qkv[0, :dim] = 0
    wq, wk = ((1 + 0.3 * torch.randn(dim, generator=g)).bfloat16() for _ in range(2))
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(4000, dtype=torch.float64)[:, None] * 250.0 * inv
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, 4000, (tokens,), generator=g).int()
    pos[-1] = 3999
    views = lambda t: (t[:, :hq * dim].unflatten(1, (hq, dim)), t[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim)))
    for weights in ((wq, wk), (None, None)):
        dev = qkv.cuda()
        args = dict(q_weight=None if weights[0] is None else wq.cuda(), k_weight=None if weights[0] is None else wk.cuda(),
                    eps=1e-6, interleaved=interleaved)
        q, k = fp8mm.qk_norm_rope(*views(dev), table.cuda(), pos.cuda(), **args)
        for x, y, w in zip(views(qkv), (q, k), weights):
            want, size = ref.norm_rope(x, w, table, pos, 1e-6, interleaved)
            assert ((y.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all()
        # in place, with padding rows
        skip = pos.clone()
        skip[::3] = -1
        fp8mm.qk_norm_rope(*views(dev), table.cuda(), skip.cuda(), q_out=views(dev)[0], k_out=views(dev)[1], **args)
        got = dev.cpu()
        assert torch.equal(got[:, (hq + hk) * dim:], qkv[:, (hq + hk) * dim:]) and torch.equal(got[::3], qkv[::3])
        keep = skip >= 0
        for x, y in zip(views(got), (q, k)):
            assert torch.equal(x[keep], y.cpu()[keep])


# ------------------------------------------------------------------ together

def test_decode_steps_from_a_projection():
    """A projection's output through norm and rotation, the cache and attention, token after token, with a fork
    and a moved page between: the same as the references over what the cache then holds."""
    hq, hk, dim, ps = 4, 2, 64, 16
    g = torch.Generator().manual_seed(77)
    ang = torch.arange(200, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    table = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    wq, wk = (torch.ones(dim).bfloat16().cuda() for _ in range(2))
    w = fp8mm.mxfp8_quantize((torch.randn((hq + 2 * hk) * dim, 256, generator=g) * 0.1).bfloat16().cuda())
    cache = ref.Cache(12, ps, hk, dim, seed=1)
    dev = cache.data.cuda()
    ws = torch.zeros(fp8mm.mxfp4_kv_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    pages = [[3, 0], [7]]
    lens = [0, 0]
    for step, new in enumerate([[20, 5], [1, 1], [1, 1, 1], [1, 1, 1]]):
        if step == 2:                                      # fork sequence 0, then move a page of sequence 1
            pages.append([pages[0][0], 9])
            lens.append(lens[0])
            fp8mm.kv_copy_pages(dev, [pages[0][1], pages[1][0]], [9, 1])
            cache.data[[9, 1]] = cache.data[[pages[0][1], pages[1][0]]]
            pages[1][0] = 1
        lens = [a + b for a, b in zip(lens, new)]
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        tab = _i32([p + [-1] * (2 - len(p)) for p in pages])
        x = torch.randn(cu[-1], 256, generator=g).bfloat16().cuda()
        qkv = fp8mm.mxfp8_gemm(*fp8mm.mxfp8_quantize(x), *w)
        q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([hq * dim, hk * dim, hk * dim], 1))
        pos = _i32(sum([list(range(n - m, n)) for n, m in zip(lens, new)], []))
        q, k = fp8mm.qk_norm_rope(q, k, table, pos, q_weight=wq, k_weight=wk)
        fp8mm.mxfp4_kv_append(k, v, dev, tab, _i32(lens), ps, cu_seqlens=_i32(cu))
        out = fp8mm.mxfp4_kv_attention(q, dev, tab, _i32(lens), ps, cu_seqlens=_i32(cu), workspace=ws)
        (kc, ke), (vc, ve) = ref.quantize(k.cpu()), ref.quantize(v.cpu())
        for s, n in enumerate(new):
            for t in range(n):
                p = lens[s] - n + t
                cache.write(pages[s][p // ps], p % ps, kc[cu[s] + t], ke[cu[s] + t], vc[cu[s] + t], ve[cu[s] + t])
        assert torch.equal(dev.cpu(), cache.data)
        _check_attention(out, None, q.cpu(), cache, pages, lens, cu, dim ** -0.5)
